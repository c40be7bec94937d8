"""GPU parity of the per-channel gated linear recurrence (gdr_scan_fwd, _bwd, _step) with its fp64
definition (oracle/block.py).

Tolerances are error bounds, element by element, from the fp64 quantities.  With u = 2^-24: the
decay a (one exponential within 3u, one sum, one reciprocal within 2u, one product: 7u), its product
with the state and the sum (2u), and in the chunked form the run's products (3u) put at most 12u of
the two terms' magnitudes into each step.  The exponent g log2(e) is one rounded product with a
rounded constant: u |g| and 0.25 u |g| in a and in 1 - a, relatively.  fp32 has no normal value
below 2^-126: a decay or 1 - a smaller than that comes out as any value up to it, so FLOOR = 2^-126
is added to their absolute errors (beyond |g| = 90 the smaller of the two is all FLOOR, and the other
one does not move).  So, with C = 12u + 1.25u min(|g|, 90) a step and what is there already carried
on by a, E_t = a_t E_{t-1} + (C a_t + FLOOR) H_{t-1} + (C w_t + FLOOR) |x_t|, with H the recurrence of
the magnitudes, bounds the error of h_t; the gradients follow by the product rule.  A 16-bit output
adds half a step."""
import numpy as np
import pytest

from oracle import block as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}
FLOOR = 2.0 ** -126
TINY = 1e-37                # results below the normal range may be flushed


@pytest.fixture(scope="module")
def G():
    from recurrent_state_memory_b200 import gdr
    gdr.lib()
    return gdr


def _dt(n):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[n]


def _walk(a, b, s0):
    """The recurrence s_t = a_t s_{t-1} + b_t: (after every token, before every token)."""
    out, before, s = np.zeros_like(a), np.zeros_like(a), s0.copy()
    for t in range(a.shape[1]):
        before[:, t] = s
        s = a[:, t] * s + b[:, t]
        out[:, t] = s
    return out, before


class Case:
    def __init__(self, B, T, D, x="bf16", g="f32", gate_mode=1, tied=False, lengths=None, h0=True, out=None, seed=0,
                 gates=None, slices=False):
        import torch
        rng = np.random.default_rng(seed + 7 * T + D)
        raw = rng.normal(size=(B, T, D)) * 2 - (1 if tied else 0)
        if gate_mode == 0:
            raw = -np.exp(raw - 2)
        if gates is not None:
            raw = np.asarray(gates)[rng.integers(0, len(gates), size=(B, T, D))]
        self.gate_mode, self.tied, self.lengths, self.out = gate_mode, tied, lengths, out or x
        t = lambda v, d: torch.from_numpy(np.asarray(v, np.float32)).to("cuda").to(_dt(d))
        self.x, self.g = t(rng.normal(size=(B, T, D)), x), t(raw, g)
        if slices:              # both as slices of one projection's output
            wide = torch.empty((B, T, 2 * D + 3), dtype=_dt(x), device="cuda").normal_()
            wide[..., 1:D + 1] = self.x
            self.x = wide[..., 1:D + 1]
            both = torch.empty((B, T, 2 * D), dtype=_dt(g), device="cuda").normal_()
            both[..., D:] = self.g
            self.g = both[..., D:]
        self.h0 = t(rng.normal(size=(B, D)), "f32") if h0 else None
        self.dh, self.dhT = t(rng.normal(size=(B, T, D)), self.out), t(rng.normal(size=(B, D)), "f32")
        self.len = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
        if lengths is not None:         # what lies behind a sequence is never read
            for b, n in enumerate(lengths):
                for v in (self.x, self.g, self.dh):
                    v[b, max(n, 0):] = float("nan")

    def kw(self):
        return dict(gate_mode=self.gate_mode, tied=self.tied, lengths=self.len)

    def wide(self):
        f = lambda v: None if v is None else np.nan_to_num(v.double().cpu().numpy(), nan=0.0, posinf=np.inf, neginf=-np.inf)
        return f(self.x), f(self.g), f(self.h0), f(self.dh), f(self.dhT)


def _near(got, ref, err, half):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape and np.all(np.isfinite(got))
    off = np.abs(got - ref) - (err + half * np.abs(ref) + TINY)
    assert off.max(initial=-1) <= 0, f"{off.max()} above the bound at {np.unravel_index(off.argmax(), off.shape)}"


def _bounds(c):
    x, g, h0, dh, dhT = c.wide()
    B, T, D = x.shape
    n = np.full(B, T) if c.lengths is None else np.clip(c.lengths, 0, T)
    inside = np.arange(T)[None] < n[:, None]
    inside = inside[..., None]
    a, rest = O.decay(g, c.gate_mode)
    a = np.where(inside, a, 1.0)
    wx = np.where(inside, np.abs(x) * (rest if c.tied else 1.0), 0.0)
    h0 = np.zeros((B, D)) if h0 is None else h0
    C = U * (12 + 1.25 * np.minimum(np.abs(g), 90))
    _, before = _walk(a, wx, np.abs(h0))
    err, err_before = _walk(a, np.where(inside, C * (a * before + wx) + FLOOR * (before + np.abs(x)), 0.0), np.zeros((B, D)))
    # the state's gradient, from the end
    rev = lambda v: v[:, ::-1]
    up = np.concatenate([np.ones((B, 1, D)), rev(a)[:, :-1]], 1)        # a_{t+1}
    mag = np.where(inside, np.abs(dh), 0.0)
    mag[:, -1] += np.abs(dhT)
    lam, _ = _walk(up, rev(mag), np.zeros((B, D)))
    Cup = np.concatenate([C[:, -1:], rev(C)[:, :-1]], 1)                # a_{t+1}'s
    lam_err, _ = _walk(up, Cup * lam + 2 * FLOOR * lam, np.zeros((B, D)))
    lam, lam_err = rev(lam), rev(lam_err)
    w = rest if c.tied else 1.0
    dx_err = np.where(inside, w * (lam_err + C * lam) + FLOOR * lam, 0.0)
    slope = np.abs(a * rest if c.gate_mode == 1 else a)
    size = before + (np.abs(x) if c.tied else 0.0)
    dg_err = np.where(inside, slope * (lam_err * size + lam * err_before + (8 * U + 2 * C) * lam * size) + 2 * FLOOR * lam * size, 0.0)
    h0_err = a[:, 0] * (lam_err[:, 0] + C[:, 0] * lam[:, 0]) + FLOOR * lam[:, 0]
    return err, err_before, dx_err, dg_err, h0_err


def _check(G, c):
    x, g, h0, dh, dhT = c.wide()
    h, hT, ckpt = G.scan_fwd(c.x, c.g, c.h0, out_dtype=_dt(c.out), want_ckpt=True, **c.kw())
    d = G.scan_bwd(c.x, c.g, ckpt, c.dh, c.dhT, **c.kw())
    assert h.dtype == _dt(c.out) and d["x"].dtype == c.x.dtype and d["g"].dtype == c.g.dtype
    err, err_before, dx_err, dg_err, h0_err = _bounds(c)
    rh, rs, before = O.scan_fwd(x, g, h0, c.gate_mode, c.tied, c.lengths)
    _near(h, rh, err, HALF[c.out])
    _near(hT, rs, err[:, -1], U)
    _near(ckpt, before[:, ::G.SCAN_CKPT], err_before[:, ::G.SCAN_CKPT], U)
    rx, rg, r0 = O.scan_bwd(x, g, h0, dh, dhT, c.gate_mode, c.tied, c.lengths)
    half = {2: HALF["bf16"], 4: U}
    _near(d["x"], rx, dx_err, half[c.x.element_size()])
    _near(d["g"], rg, dg_err, half[c.g.element_size()])
    _near(d["h0"], r0, h0_err, U)
    assert G.query_device_status() == G.GDR_OK


@pytest.mark.parametrize("T", [1, 2, 31, 63, 64, 65, 127, 128, 129, 255, 257, 700])
@pytest.mark.parametrize("D", [1, 63, 64, 68])
def test_lengths_and_channels(G, T, D):
    _check(G, Case(2, T, D, gate_mode=T % 2, tied=D % 2 == 1))


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("g", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("D", [72, 77])
def test_types(G, x, g, out, D):
    _check(G, Case(2, 150, D, x=x, g=g, out=out, tied=True))


@pytest.mark.parametrize("gate_mode", [0, 1])
@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("h0", [False, True])
def test_modes(G, gate_mode, tied, h0):
    _check(G, Case(3, 400, 40, x="f32", gate_mode=gate_mode, tied=tied, h0=h0))


@pytest.mark.parametrize("D", [64, 61])
@pytest.mark.parametrize("lengths", [[300, 0, 1, 64], [5, 299, 128, 129], [-7, 1000, 65, 192]])
def test_ragged_batches(G, lengths, D):
    """Empty, one-token and full sequences; lengths outside 0 .. T are clamped; NaN behind each."""
    _check(G, Case(4, 300, D, lengths=[n for n in lengths], x="f32"))


@pytest.mark.parametrize("D", [64, 48, 33])
def test_slices_of_a_projection(G, D):
    _check(G, Case(2, 200, D, x="bf16", g="bf16", slices=True))


@pytest.mark.parametrize("D", [64, 30])
def test_tensors_that_start_on_no_16_bytes(G, D):
    """Contiguous x, g, dh, h0 and step states at odd places of larger tensors."""
    import torch
    c = Case(2, 150, D)

    def moved(v):
        flat = torch.empty(v.numel() + 1, dtype=v.dtype, device="cuda")
        flat[1:] = v.reshape(-1)
        return flat[1:].view(v.shape)

    c.x, c.g, c.dh, c.h0, c.dhT = map(moved, (c.x, c.g, c.dh, c.h0, c.dhT))
    assert c.x.data_ptr() % 4 and c.x.is_contiguous()
    _check(G, c)
    s, ref = moved(c.h0), c.h0.clone()
    o = G.scan_step(c.x[:, 0], c.g[:, 0], s)
    assert torch.equal(o, G.scan_step(c.x[:, 0].contiguous(), c.g[:, 0].contiguous(), ref)) and torch.equal(s, ref)


@pytest.mark.parametrize("gate_mode,gates", [(1, [-np.inf, np.inf, 90.0, -90.0, 200.0, 0.0, -17.0]),
                                             (0, [-np.inf, 0.0, -1e-9, -100.0, -1e30, -0.5])])
@pytest.mark.parametrize("tied", [False, True])
def test_gates_at_the_ends(G, gate_mode, gates, tied):
    """Gates that keep all, keep nothing, and beyond the exponential's range."""
    _check(G, Case(1, 260, 64, x="f32", gate_mode=gate_mode, gates=gates, tied=tied))


def test_long_sequences_of_few_channels(G):
    _check(G, Case(1, 6000, 4, x="f32", g="f32", gate_mode=0))
    _check(G, Case(1, 5000, 3, x="bf16", g="bf16", tied=True))


def test_without_gradients_of_the_outputs(G):
    """dh or dh_T None is zero; dh0 may be left out."""
    import torch
    c = Case(2, 100, 20, x="f32")
    _, _, ck = G.scan_fwd(c.x, c.g, c.h0, want_ckpt=True, **c.kw())
    z = torch.zeros_like
    for dh, dhT in ((None, c.dhT), (c.dh, None), (None, None)):
        a = G.scan_bwd(c.x, c.g, ck, dh, dhT, want_dh0=False, **c.kw())
        b = G.scan_bwd(c.x, c.g, ck, z(c.dh) if dh is None else dh, z(c.dhT) if dhT is None else dhT, **c.kw())
        assert a["h0"] is None and torch.equal(a["x"], b["x"]) and torch.equal(a["g"], b["g"])


def test_backward_against_a_difference_of_the_forward(G):
    """The loss's change along one direction, in fp32 with a central step: the truncation is below
    eps^2 and the loss's own rounding below 1e-6 of its terms over the step."""
    import torch
    c = Case(2, 300, 24, x="f32", tied=True)
    _, _, ck = G.scan_fwd(c.x, c.g, c.h0, want_ckpt=True, **c.kw())
    d = G.scan_bwd(c.x, c.g, ck, c.dh, c.dhT, **c.kw())
    rng = torch.Generator("cuda").manual_seed(5)
    dirs = [torch.randn(v.shape, generator=rng, device="cuda") for v in (c.x, c.g, c.h0)]

    def loss(s):
        h, hT = G.scan_fwd(c.x + s * dirs[0], c.g + s * dirs[1], c.h0 + s * dirs[2], **c.kw())
        return (h.double() * c.dh.double()).sum() + (hT.double() * c.dhT.double()).sum()

    eps = 1e-2
    num = (loss(eps) - loss(-eps)) / (2 * eps)
    ana = sum((a.double() * b.double()).sum() for a, b in zip((d["x"], d["g"], d["h0"]), dirs))
    scale = sum((a.double() * b.double()).square().sum() for a, b in zip((d["x"], d["g"], d["h0"]), dirs)).sqrt()
    assert abs(num - ana) < 2e-2 * scale


def test_the_state_may_be_updated_in_place(G):
    import ctypes
    import torch
    c = Case(2, 333, 70, x="f32")
    h, hT = G.scan_fwd(c.x, c.g, c.h0, **c.kw())
    s, h2 = c.h0.clone(), torch.empty_like(h)
    desc = G.scan_desc(2, 333, 70, c.x.dtype, c.g.dtype, h2.dtype)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    assert G.lib().gdr_scan_fwd(desc, p(c.x), p(c.g), p(s), None, p(h2), p(s), None, None) == G.GDR_OK
    torch.cuda.synchronize()
    assert torch.equal(s, hT) and torch.equal(h, h2)


@pytest.mark.parametrize("N,D", [(1, 1), (3, 7), (5, 64), (64, 1000), (700, 33)])
@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("gt", ["f32", "bf16"])
def test_step_equals_the_forward(G, N, D, tied, gt):
    """Token by token: the outputs meet the forward's bound, and the state of a whole sequence."""
    c = Case(N, 6, D, g=gt, tied=tied)
    x, g, h0, _, _ = c.wide()
    s = c.h0.clone()
    ref, last, _ = O.scan_fwd(x, g, h0, c.gate_mode, tied)
    err = _bounds(c)[0]
    for t in range(6):
        o = G.scan_step(c.x[:, t].contiguous() if N % 2 else c.x[:, t], c.g[:, t], s, gate_mode=c.gate_mode, tied=tied)
        _near(o, ref[:, t], err[:, t], HALF["bf16"])
    _near(s, last, err[:, -1], U)


def test_very_many_sequences(G):
    """More sequences than a grid's third dimension holds: the same as in two halves."""
    import torch
    gen = torch.Generator("cuda").manual_seed(9)
    x, g = torch.randn(2, 70001, 3, 5, generator=gen, device="cuda")
    h, hT, ck = G.scan_fwd(x, g, want_ckpt=True)
    a, b = G.scan_fwd(x[:35000], g[:35000]), G.scan_fwd(x[35000:], g[35000:])
    assert torch.equal(h, torch.cat([a[0], b[0]])) and torch.equal(hT, torch.cat([a[1], b[1]]))
    d = G.scan_bwd(x, g, ck, h)
    e = G.scan_bwd(x[35000:], g[35000:], ck[35000:], h[35000:])
    assert torch.equal(d["x"][35000:], e["x"]) and torch.equal(d["g"][35000:], e["g"])
    s, o = hT.clone(), G.scan_step(x[:, 0], g[:, 0], hT)
    assert torch.equal(o, G.scan_fwd(x[:, :1].contiguous(), g[:, :1].contiguous(), s)[0][:, 0])


def test_no_tokens_no_sequences(G):
    import torch
    x = torch.empty((3, 0, 8), device="cuda")
    h0 = torch.randn(3, 8, device="cuda")
    h, hT, ck = G.scan_fwd(x, x, h0, want_ckpt=True)
    assert h.shape == (3, 0, 8) and ck.shape == (3, 0, 8) and torch.equal(hT, h0)
    assert torch.equal(G.scan_fwd(x, x)[1], torch.zeros_like(h0))
    d = G.scan_bwd(x, x, ck, x, h0)
    assert torch.equal(d["h0"], h0) and d["x"].shape == x.shape
    e = torch.empty((0, 5, 8), device="cuda")
    assert G.scan_fwd(e, e)[0].shape == (0, 5, 8)
    assert G.scan_step(e[:, 0], e[:, 0], torch.empty((0, 8), device="cuda")).shape == (0, 8)


def test_the_same_twice_on_another_stream_and_in_a_graph(G):
    import torch
    c = Case(3, 1500, 130, lengths=[1500, 700, 0])
    run = lambda: (lambda f: (*f, *G.scan_bwd(c.x, c.g, f[2], c.dh, c.dhT, **c.kw()).values()))(
        G.scan_fwd(c.x, c.g, c.h0, want_ckpt=True, **c.kw()))
    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    keep = c.x.clone()
    c.x.zero_()
    graph.replay()
    c.x.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, held))
