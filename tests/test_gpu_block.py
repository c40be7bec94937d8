"""The operators around the delta rule run together, as a recurrent block uses them: norm, scan and
their gradients through a training step; a prompt's final states, steps, beam selection and the
states that follow it in a serving loop (beside decode_step's)."""
import numpy as np
import pytest

from oracle import block as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def G():
    from recurrent_state_memory_b200 import gdr
    gdr.lib()
    return gdr


def test_a_training_step(G):
    """y = norm(x), h = scan(y, g), loss = <dh, h> + <dh_T, h_T>: every gradient against fp64, in fp32.
    The gates are near zero raw (a about 1/2), so at most a few steps' roundings add up; 1e-5 of each
    gradient's largest value is 160 u, over the 12 u a step times two of the scan's tests."""
    import torch
    B, T, D = 2, 300, 96
    gen = torch.Generator("cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x, g, w, b, h0, dh, dhT = r(B, T, D), r(B, T, D), 1 + 0.2 * r(D), 0.2 * r(D), r(B, D), r(B, T, D), r(B, D)
    n = torch.tensor([T, 123], dtype=torch.int32, device="cuda")
    y, mean, rstd = G.layernorm_fwd(x, w, b)
    h, hT, ck = G.scan_fwd(y, g, h0, tied=True, lengths=n, want_ckpt=True)
    d = G.scan_bwd(y, g, ck, dh, dhT, tied=True, lengths=n)
    e = G.layernorm_bwd(x, d["x"], mean, rstd, w)
    X, GT, W, BI, H0, DH, DT = (v.double().cpu().numpy() for v in (x, g, w, b, h0, dh, dhT))
    Y = O.layernorm_fwd(X, W, BI)[0]
    rh, rs, _ = O.scan_fwd(Y, GT, H0, 1, True, [T, 123])
    dy, dg, d0 = O.scan_bwd(Y, GT, H0, DH, DT, 1, True, [T, 123])
    dx, dw, db = O.layernorm_bwd(X, dy, W)
    for got, ref in ((h, rh), (hT, rs), (d["g"], dg), (d["h0"], d0), (e["x"], dx), (e["weight"], dw), (e["bias"], db)):
        assert np.max(np.abs(got.double().cpu().numpy() - ref)) <= 1e-5 * np.max(np.abs(ref))


def test_a_serving_loop_with_beams(G):
    """3 requests of 4 beams: the prompt's states are shared by a request's beams, then 6 tokens of
    step, selection and reorder, for the scan's states of two layers and a delta-rule layer's.  The
    selection is checked on the logits that the loop has; the states against fp64 along the chosen
    parents, which the loop must have followed exactly."""
    import torch
    R, K, D, V, T = 3, 4, 64, 501, 70
    gen = torch.Generator("cuda").manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    emb_x, emb_g, head = r(V, D), r(V, D), r(D, V) * 0.5
    prompt = r(R, T, D)
    _, hT = G.scan_fwd(prompt, prompt, tied=True)
    N = R * K
    h = hT.repeat_interleave(K, 0).expand(2, N, D).contiguous()         # two layers in one tensor
    ref = h.double().cpu().numpy().copy()
    S = torch.zeros(N, 2, 32, 32, device="cuda")                        # a delta-rule layer's states
    ref_S = S.clone()
    scores = torch.full((R, K), -float("inf"), device="cuda")
    scores[:, 0] = 0
    finished = torch.zeros((R, K), dtype=torch.bool, device="cuda")
    token = torch.zeros((R, K), dtype=torch.long, device="cuda")
    for step in range(6):
        x, g = emb_x[token.view(-1)], emb_g[token.view(-1)]
        o = G.scan_step(x, g, h[0], tied=True, out_dtype=torch.float32)
        o = G.scan_step(o, g, h[1], tied=True, out_dtype=torch.float32)
        q = x.view(N, 2, 32)
        beta = torch.full((N, 2), 0.5, device="cuda")
        G.decode_step(q, q, q, q, beta, S, qk_l2norm=True)
        G.decode_step(q, q, q, q, beta, ref_S, qk_l2norm=True)
        a, rest = O.decay(g.cpu().numpy(), 1)
        ref[0] = a * ref[0] + rest * x.double().cpu().numpy()
        ref[1] = a * ref[1] + rest * ref[0]
        logits = (o @ head).view(R, K, V)
        before = scores.clone()
        scores, parent, tok = G.beam_select(logits, scores, finished=finished, eos=7)
        rs, rp, rt = O.beam_select(logits.double().cpu().numpy(), before.cpu().numpy(), K, finished.cpu().numpy(), 7)
        assert np.array_equal(parent.cpu().numpy(), rp) and np.array_equal(tok.cpu().numpy(), rt)
        G.state_reorder(h, parent, layers=True)
        G.state_reorder(S, parent)
        ref = O.state_reorder(ref, rp, layers=True)
        flat = (torch.arange(R, device="cuda")[:, None] * K + parent).view(-1)
        ref_S = ref_S[flat].contiguous()
        finished = finished.gather(1, parent.long()) | (tok == 7)
        token = tok.long()
        assert torch.equal(S, ref_S)
        # both layers, at most 6 + 70 tokens of 12 u each of values below 10
        assert np.max(np.abs(h.double().cpu().numpy() - ref)) < 2 * 76 * 12 * U * 10
    assert G.query_device_status() == G.GDR_OK
