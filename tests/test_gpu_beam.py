"""GPU parity of the beam selection and the state reorder (gdr_beam_select, gdr_state_reorder) with
their fp64 definitions: beams and tokens are equal, scores within the fp32 sum's error, 8e-6 (with
u = 2^-24: exponents d off by 2.25 u |d|, |d| at most log V <= 12 in the weighted mean, 27 u; the
exponentials 3 u; 48 sums 48 u; 78 u = 4.7e-6 of the sum and so of its logarithm) and half a step."""
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


def _dt(n):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[n]


def _check(G, logits, scores, M, finished=None, eos=0):
    import torch
    s, p, t = G.beam_select(logits, scores, M, finished=finished, eos=eos)
    assert s.shape == p.shape == t.shape == (logits.shape[0], M if M else logits.shape[1])
    f = lambda v: None if v is None else v.cpu().numpy()
    rs, rp, rt = O.beam_select(logits.double().cpu().numpy(), f(scores), s.shape[1], f(finished), eos)
    assert np.array_equal(p.cpu().numpy(), rp)
    assert np.array_equal(t.cpu().numpy(), rt)
    s = s.double().cpu().numpy()
    live = np.isfinite(rs)
    assert np.array_equal(live, np.isfinite(s)) and np.array_equal(s[~live], rs[~live])
    assert np.all(np.abs(s - rs)[live] <= 8e-6 + U * np.abs(rs)[live])


def _make(g, k, v, x="f32", seed=0, std=2.5, banned=0.02):
    import torch
    gen = torch.Generator("cuda").manual_seed(seed + v)
    z = torch.randn((g, k, v), generator=gen, device="cuda") * std
    if banned:
        z[torch.rand((g, k, v), generator=gen, device="cuda") < banned] = -float("inf")
    return z.to(_dt(x)), torch.randn((g, k), generator=gen, device="cuda") * 1.5 - 20


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("v", [1, 2, 7, 31, 32, 64, 255, 256, 257, 1000, 2047, 2048, 2049, 8192, 8193, 20011, 65537])
def test_vocabularies(G, x, v):
    k = 4
    _check(G, *_make(3, k, v, x), min(k, k * v))


@pytest.mark.parametrize("k", [1, 2, 3, 8, 16, 33, 64])
@pytest.mark.parametrize("m", [1, 5, 16, 64])
def test_beams_and_candidates(G, k, m):
    _check(G, *_make(2, k, 300, "bf16" if k % 2 else "f32", seed=m), m)


@pytest.mark.parametrize("v", [10, 5000])
@pytest.mark.parametrize("m", [3, 40])
def test_everything_is_equal(G, v, m):
    """All candidates tie: the lowest k * V + v, in order."""
    import torch
    _check(G, torch.zeros((2, 4, v), device="cuda"), torch.full((2, 4), -3.0, device="cuda"), m)


def test_twin_beams_tie(G):
    """Equal rows and scores: every candidate ties with its twin; the first beam goes first."""
    z, s = _make(3, 1, 3001)
    _check(G, z.expand(3, 5, 3001).contiguous(), s.expand(3, 5).contiguous(), 12)


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_neighbours_closer_than_the_fp32_sum(G, x):
    """Beams whose best candidates differ by 1e-7 of the score: the order is the 64-bit one."""
    import torch
    for seed in range(6):
        z, _ = _make(1, 6, 4000, x, seed=100 + seed, banned=0)
        best = z.double().log_softmax(2).amax(2)
        s = (-10 - best).float()                # all beams' best land near -10, as near as fp32 scores can
        s += (torch.randperm(6, device="cuda")[None] - 3) * 1e-6
        _check(G, z, s, 6)


def test_quantised_scores_with_many_ties(G):
    import torch
    z = torch.randint(-4, 5, (3, 6, 2500), device="cuda").float()
    _check(G, z, torch.randint(-2, 1, (3, 6), device="cuda").float(), 48)


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_ascending_and_descending_rows(G, x):
    import torch
    up = torch.linspace(-9, 9, 9000, device="cuda").expand(2, 2, 9000).contiguous().to(_dt(x))
    s = torch.tensor([[-1.0, -1.5], [-2.0, -1.0]], device="cuda")
    _check(G, up, s, 20)
    _check(G, up.flip(2).contiguous(), s, 20)


def test_masked_beams(G):
    """-inf and lowest values, a beam with one token left, beams with none, more candidates than tokens."""
    import torch
    z, s = _make(2, 5, 700, seed=3)
    z[0, 0] = -float("inf")
    z[0, 1] = -float("inf")
    z[0, 1, 345] = 1.0
    z[0, 2] = torch.finfo(torch.float32).min
    z[1, :] = -float("inf")
    z[1, 3, 699] = -5.0
    _check(G, z, s, 9)
    _check(G, z[1:].contiguous(), s[1:].contiguous(), 64)


def test_poisoned_beams_drop_out(G):
    z, s = _make(2, 5, 900, seed=4)
    z[0, 0, 17] = float("nan")
    z[0, 1, 899] = float("inf")
    s[0, 2] = float("nan")
    s[1, 0] = -float("inf")
    s[1, 3] = float("inf")
    _check(G, z, s, 10)
    s[0, 3:] = -float("inf")
    _check(G, z, s, 10)                # no candidate is left in the first group


def test_finished_beams(G):
    import torch
    z, s = _make(4, 4, 1234, seed=5)
    s += torch.rand_like(s) * 12
    f = torch.tensor([[1, 0, 0, 1], [0, 0, 0, 0], [1, 1, 1, 1], [0, 1, 0, 0]], dtype=torch.bool, device="cuda")
    for eos in (0, 2, 1233):
        _check(G, z, s, 4, f, eos)
        _check(G, z, s, 8, f, eos)
    s[2, 1] = -float("inf")
    _check(G, z, s, 6, f, 1)


def test_the_first_token(G):
    import torch
    z, s = _make(3, 8, 5000, "bf16", seed=6)
    z = z[:, :1].expand(3, 8, 5000).contiguous()
    s.fill_(-float("inf"))
    s[:, 0] = 0
    _check(G, z, s, 16)


def test_padded_vocabulary_rows(G):
    """Logits as slices of wider rows; what lies behind V is not read."""
    import torch
    for x, v, row in (("bf16", 1000, 1024), ("f32", 999, 1001), ("bf16", 4001, 4008)):
        z, s = _make(2, 3, v, x, seed=7)
        wide = torch.full((2, 3, row), float("nan"), device="cuda", dtype=z.dtype)
        wide[..., :v] = z
        _check(G, wide[..., :v], s, 6)


def test_flat_and_far_logits(G):
    """Large vocabularies of near-equal logits (all mass in the sum), and logits in the thousands."""
    import torch
    z, s = _make(1, 3, 150000, "f32", std=1e-3, banned=0)
    _check(G, z, s, 8)
    z, s = _make(2, 3, 777, "f32", std=3000.0, banned=0)
    _check(G, z, s, 8)


def test_selection_twice_on_a_stream_and_in_graphs(G):
    """Two captured graphs replayed at once on two streams keep apart."""
    import torch
    a, b = _make(8, 4, 20000, "bf16", seed=8), _make(8, 4, 20000, "bf16", seed=9)
    first = [G.beam_select(*v, 8) for v in (a, b)]
    graphs, held = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for gr, v in zip(graphs, (a, b)):
        with torch.cuda.graph(gr):
            held.append(G.beam_select(*v, 8))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for f, h in zip(first, held):
        assert all(torch.equal(x, y) for x, y in zip(f, h))


def test_very_many_groups(G):
    """More beams than a grid's second dimension holds; every group by the definition's top-1."""
    import torch
    z, s = _make(40000, 2, 40, "bf16", seed=11, banned=0)
    sc, p, t = G.beam_select(z, s, 1)
    c = (z.double().log_softmax(2) + s.double()[..., None]).view(40000, 80)
    top = c.topk(2, dim=1)
    at = p[:, 0].long() * 40 + t[:, 0].long()
    assert torch.equal(c.gather(1, at[:, None]), top.values[:, :1])
    clear = top.values[:, 0] > top.values[:, 1]
    assert torch.equal(at[clear], top.indices[:, 0][clear])


# ---------------------------------------------------------------- reorder ----


@pytest.mark.parametrize("k", [1, 2, 3, 4, 5, 8, 11, 16, 17, 64])
@pytest.mark.parametrize("e,dt", [(1, "f32"), (3, "f32"), (4, "f32"), (1022, "f32"), (2048, "f32"), (7, "bf16"),
                                  (2, "bf16"), (4096, "bf16")])
def test_reorder(G, k, e, dt):
    import torch
    gen = torch.Generator("cuda").manual_seed(k * 100 + e)
    for L, g in ((1, 1), (3, 4)):
        S = torch.randn((L, g * k, e), generator=gen, device="cuda").to(_dt(dt))
        p = torch.randint(0, k, (g, k), generator=gen, device="cuda", dtype=torch.int32)
        ref = O.state_reorder(S.float().cpu().numpy(), p.cpu().numpy(), layers=True)
        assert G.state_reorder(S, p, layers=True) is S
        assert np.array_equal(S.float().cpu().numpy(), ref)
    assert G.query_device_status() == G.GDR_OK


@pytest.mark.parametrize("kind", ["self", "swap", "rotate", "one", "reverse"])
def test_reorder_of_cycles(G, kind):
    import torch
    k = 8
    j = torch.arange(k)
    p = {"self": j, "swap": j ^ 1, "rotate": (j + 1) % k, "one": j * 0 + 5, "reverse": k - 1 - j}[kind]
    p = p.int().expand(3, k).contiguous().cuda()
    S = torch.randn(3 * k, 2, 16, 130, device="cuda")
    ref = O.state_reorder(S.cpu().numpy(), p.cpu().numpy())
    G.state_reorder(S, p)
    assert np.array_equal(S.cpu().numpy(), ref)


def test_reorder_of_one_byte_states_and_bad_parents(G):
    """A parent outside the group keeps its beam's state and sets the status word, once."""
    import torch
    S = torch.arange(12, dtype=torch.uint8, device="cuda")
    p = torch.tensor([[1, 7, 0, -1], [3, 3, 2, 0], [0, 1, 2, 4]], dtype=torch.int32, device="cuda")
    ref = O.state_reorder(S.cpu().numpy(), p.cpu().numpy())
    G.state_reorder(S, p)
    assert np.array_equal(S.cpu().numpy(), ref)
    assert G.query_device_status() == G.GDR_ERR_INDEX
    assert G.query_device_status() == G.GDR_OK


def test_reorder_of_very_many_groups(G):
    import torch
    S = torch.randn(3, 140000, 5, device="cuda")
    p = torch.randint(0, 2, (70000, 2), device="cuda", dtype=torch.int32)
    at = (torch.arange(70000, device="cuda")[:, None] * 2 + p).view(-1)
    ref = S[:, at]
    G.state_reorder(S, p, layers=True)
    assert torch.equal(S, ref)


def test_reorder_at_any_alignment(G):
    import torch
    for dt, at in ((torch.uint8, 3), (torch.bfloat16, 1), (torch.float32, 1), (torch.float32, 2)):
        S = torch.randint(0, 100, (8 * 64 + at,), device="cuda").to(dt)[at:].view(8, 64)
        p = torch.tensor([[3, 0, 0, 2], [1, 1, 2, 0]], dtype=torch.int32, device="cuda")
        ref = O.state_reorder(S.float().cpu().numpy(), p.cpu().numpy())
        G.state_reorder(S, p)
        assert np.array_equal(S.float().cpu().numpy(), ref)


def test_reorder_of_nothing(G):
    import torch
    G.state_reorder(torch.empty((0, 5), device="cuda"), torch.empty((0, 4), dtype=torch.int32, device="cuda"))
    G.state_reorder(torch.empty((8, 0), device="cuda"), torch.zeros((2, 4), dtype=torch.int32, device="cuda"))


def test_reorder_past_32_bits(G):
    """States behind byte 2^33: 40 beams of 256 MB."""
    import torch
    S = torch.empty((40, 1 << 26), dtype=torch.float32, device="cuda")
    S[:] = torch.arange(40.0, device="cuda")[:, None]
    p = torch.tensor([[7, 6, 5, 4, 3, 2, 1, 0]] * 5, dtype=torch.int32, device="cuda")
    G.state_reorder(S, p)
    want = torch.arange(40.0, device="cuda").view(5, 8).flip(1).reshape(-1)
    assert torch.equal(S[:, 0], want) and torch.equal(S[:, -1], want) and torch.equal(S[:, 12345678], want)
