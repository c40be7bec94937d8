"""GPU parity of the layer norm and its gradient (gdr_layernorm_fwd, _bwd) with the fp64 definition.

Tolerances: bounds from the fp64 quantities, u = 2^-24.  A sum of n terms in fp32 is off by at most
n u times the sum of their magnitudes in any order; S = D + 8 stands for a row's sums.  The mean is
off by S u mean|x|, which moves x hat by rstd times that (and the centred values by their own
rounding); the variance is formed from the centred values, so rstd is off by S u of itself, plus
the mean's error squared.  A 16-bit output adds half a step."""
import numpy as np
import pytest

from oracle import block as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


@pytest.fixture(scope="module")
def G():
    from recurrent_state_memory_b200 import gdr
    gdr.lib()
    return gdr


def _dt(n):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[n]


def _near(got, ref, err, half):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape and np.all(np.isfinite(got))
    off = np.abs(got - ref) - (err + half * np.abs(ref) + 1e-37)
    assert off.max(initial=-1) <= 0, f"{off.max()} above the bound at {np.unravel_index(off.argmax(), off.shape)}"


def _check(G, rows, D, x="bf16", y=None, w="f32", weight=True, bias=True, offset=0.5, eps=1e-5):
    import torch
    rng = np.random.default_rng(rows + 31 * D)
    y = y or x
    t = lambda v, d: torch.from_numpy(np.asarray(v, np.float32)).to("cuda").to(_dt(d))
    xs = t(rng.normal(size=(rows, D)) * np.exp(0.5 * rng.normal(size=(rows, 1))) + offset * rng.normal(size=(rows, 1)), x)
    ws = t(1 + 0.3 * rng.normal(size=D), w) if weight else None
    bs = t(0.3 * rng.normal(size=D), w) if bias else None
    dy = t(rng.normal(size=(rows, D)), y)
    f = lambda v: None if v is None else v.double().cpu().numpy()
    out, mean, rstd = G.layernorm_fwd(xs, ws, bs, eps=eps, out_dtype=_dt(y))
    X, W, B, DY = f(xs), f(ws), f(bs), f(dy)
    ry, rm, rr = O.layernorm_fwd(X, W, B, eps)
    S = (D + 8) * U
    aw = 1.0 if W is None else np.abs(W)
    merr = S * np.abs(X).mean(-1)
    hat = np.abs((X - rm[:, None]) * rr[:, None])
    rerr = S + (rr * merr) ** 2 + 4 * U                                  # relative
    herr = rr[:, None] * merr[:, None] + (rerr[:, None] + 3 * U) * hat   # of x hat
    _near(mean, rm, merr, U)
    _near(rstd, rr, rerr * rr, U)
    _near(out, ry, aw * herr + 2 * U * (np.abs(ry) + (0 if B is None else np.abs(B))), HALF[y])
    d = G.layernorm_bwd(xs, dy, mean, rstd, ws, with_bias=bias)
    rx, rw, rb = O.layernorm_bwd(X, DY, W, eps)
    wd = np.abs(DY) * aw
    c1, c2 = wd.mean(-1, keepdims=True), (wd * hat).mean(-1, keepdims=True)
    c2err = (wd * herr).mean(-1, keepdims=True) + S * c2
    xerr = rr[:, None] * (S * c1 + herr * c2 + hat * c2err + (rerr[:, None] + 6 * U) * (wd + c1 + hat * c2))
    _near(d["x"], rx, xerr, HALF[x])
    R = (rows + 8) * U
    if weight:
        _near(d["weight"], rw, (np.abs(DY) * (herr + R * hat)).sum(0), U)
    else:
        assert d["weight"] is None
    if bias:
        _near(d["bias"], rb, R * np.abs(DY).sum(0), U)
    else:
        assert d["bias"] is None


@pytest.mark.parametrize("D", [1, 2, 3, 8, 16, 31, 32, 33, 64, 96, 100, 128, 192, 250, 256, 257, 512, 640, 1000, 1024,
                               1025, 1536, 2047, 2048, 2056, 4096, 5000, 8192, 8200, 16384, 20000])
def test_widths(G, D):
    _check(G, 7, D)


@pytest.mark.parametrize("D", [1, 5, 64, 128, 333, 1000, 2048, 9001])
def test_widths_in_32_bits(G, D):
    _check(G, 5, D, x="f32")


@pytest.mark.parametrize("x,y", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("D,rows", [(8200, 1), (9000, 160), (12288, 7), (16384, 330)])
def test_wide_rows(G, x, y, D, rows):
    _check(G, rows, D, x=x, y=y)
    if rows == 7:
        _check(G, rows, D, x=x, y=y, weight=False)
        _check(G, rows, D, x=x, y=y, weight=False, bias=False)


def test_the_widest_rows(G):
    _check(G, 2, 70001, x="f32")
    _check(G, 3, 131072)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 149, 1000, 5003])
@pytest.mark.parametrize("D", [64, 128, 77])
def test_rows(G, rows, D):
    _check(G, rows, D)


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("y", ["bf16", "f32"])
@pytest.mark.parametrize("w", ["bf16", "f32"])
@pytest.mark.parametrize("D", [136, 1029, 2600])
def test_types(G, x, y, w, D):
    _check(G, 21, D, x=x, y=y, w=w)


@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("D", [128, 3001])
def test_optional_weights(G, weight, bias, D):
    _check(G, 40, D, weight=weight, bias=bias)


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_tensors_that_start_on_no_16_bytes(G, x):
    """Contiguous slices of larger tensors: the results are those of copies (other loads, the same
    order of sums within a row up to the lanes' split, so within the tests' bounds of each other)."""
    import torch
    gen = torch.Generator("cuda").manual_seed(3)
    flat = torch.randn(2 * 40 * 96 + 2, generator=gen, device="cuda").to(_dt(x))
    a, dy = flat[1:1 + 40 * 96].view(40, 96), flat[2 + 40 * 96:].view(40, 96)
    w = torch.randn(97, generator=gen, device="cuda")[1:]
    y, m, r = G.layernorm_fwd(a, w)
    d = G.layernorm_bwd(a, dy, m, r, w)
    y2, m2, r2 = G.layernorm_fwd(a.clone(), w.clone())
    d2 = G.layernorm_bwd(a.clone(), dy.clone(), m2, r2, w.clone())
    for got, ref in ((y, y2), (m, m2), (r, r2), (d["x"], d2["x"]), (d["weight"], d2["weight"]), (d["bias"], d2["bias"])):
        scale = ref.double().abs().max()
        assert (got.double() - ref.double()).abs().max() <= (2.0 ** -7 if got.dtype == torch.bfloat16 else 200 * U) * scale


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("D", [9, 10, 12, 13, 17, 33, 65, 129, 249, 333, 514, 761, 1025, 1530, 2052, 5001])
@pytest.mark.parametrize("rows", [1, 2, 3, 9, 1201])
def test_rows_that_start_anywhere(G, x, D, rows):
    """Widths that are no multiple of 16 bytes: rows begin and end inside one."""
    _check(G, rows, D, x=x)


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("D,rows", [(9, 50), (12, 33), (33, 21), (333, 11), (514, 9), (1025, 17), (5001, 10)])
def test_rows_end_where_they_end(G, x, D, rows):
    """Tensors inside of larger ones: what lies around them is neither used nor written, and rows of
    NaN and infinities stay out of their neighbours."""
    import ctypes

    import torch
    t, gen, n = _dt(x), torch.Generator("cuda").manual_seed(D), rows * D

    def inside(fill):
        whole = torch.full((n + 128,), fill, device="cuda", dtype=t)
        return whole, whole[64:64 + n].view(rows, D)

    _, a = inside(float("nan"))
    _, dy = inside(float("inf"))
    a.copy_(torch.randn(rows, D, generator=gen, device="cuda"))
    dy.copy_(torch.randn(rows, D, generator=gen, device="cuda"))
    w = torch.randn(D, generator=gen, device="cuda")
    desc = G.norm_desc(rows, D, t, t)
    lib, ptr = G.lib(), lambda v: ctypes.c_void_p(v.data_ptr())
    flt = lambda v: ctypes.cast(ptr(v), ctypes.POINTER(ctypes.c_float))
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def run():
        (wy, y), (wx, dx) = inside(7.0), inside(7.0)
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        assert lib.gdr_layernorm_fwd(ctypes.byref(desc), ptr(a), ptr(w), None, ptr(y), flt(mean), flt(rstd), st) == 0
        assert lib.gdr_layernorm_bwd(ctypes.byref(desc), ptr(a), ptr(dy), ptr(w), flt(mean), flt(rstd), ptr(dx), None, None,
                                     None, 0, st) == 0
        for whole in (wy, wx):
            assert (whole[:64] == 7).all() and (whole[64 + n:] == 7).all()
        return y, dx

    ref = run()
    assert all(torch.isfinite(v).all() for v in ref)
    bad = rows // 2
    a[bad], dy[bad] = float("inf"), float("nan")
    keep = [r for r in range(rows) if r != bad]
    for got, want in zip(run(), ref):
        assert torch.equal(got[keep], want[keep]) and torch.isnan(got[bad]).all()


def test_rows_far_from_zero(G):
    """A row's offset is a hundred times its spread: the variance comes from the centred values."""
    _check(G, 30, 512, x="f32", offset=100.0)


@pytest.mark.parametrize("D", [128, 2048])
def test_constant_rows(G, D):
    """No spread: y is the bias, rstd 1 / sqrt(eps), dx the centred w dy."""
    import torch
    x = torch.full((4, D), 3.0, device="cuda")
    w, b = torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    y, mean, rstd = G.layernorm_fwd(x, w, b, eps=1e-4)
    assert torch.equal(y, b.expand(4, D)) and torch.equal(mean, torch.full((4,), 3.0, device="cuda"))
    assert torch.allclose(rstd, torch.full((4,), 100.0, device="cuda"), rtol=4e-7)


def test_a_row_of_nan_stays_in_its_row(G):
    import torch
    x = torch.randn(9, 256, device="cuda")
    ref = G.layernorm_fwd(x)[0]
    x[4, 17] = float("nan")
    x[6, 3] = float("inf")
    y = G.layernorm_fwd(x)[0]
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(y[keep], ref[keep]) and torch.isnan(y[4]).all() and torch.isnan(y[6]).any()


def test_many_rows_sum_in_a_fixed_order(G):
    """B4 T512 H16 rows of 128 as [.., D]: the same bits twice, on another stream and in a graph."""
    import torch
    x = torch.randn(4, 512, 16, 128, device="cuda").bfloat16()
    dy = torch.randn_like(x)
    w = torch.randn(128, device="cuda")
    _, mean, rstd = G.layernorm_fwd(x, w)
    assert mean.shape == (4, 512, 16)
    run = lambda: list(G.layernorm_bwd(x, dy, mean, rstd, w).values())
    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(first, again, held))
    ref = O.layernorm_bwd(x.double().cpu().numpy(), dy.double().cpu().numpy(), w.double().cpu().numpy())
    scale = np.sqrt(x.numel() / 128)        # 32768 rows of unit terms: their sum's standard deviation
    for got, r in zip(first[1:], ref[1:]):
        assert np.max(np.abs(got.double().cpu().numpy() - r)) < 32768 * U * 4 * scale


def test_parts_of_the_gradient(G):
    import torch
    x, dy = torch.randn(100, 300, device="cuda"), torch.randn(100, 300, device="cuda")
    w = torch.randn(300, device="cuda")
    _, m, r = G.layernorm_fwd(x, w)
    full = G.layernorm_bwd(x, dy, m, r, w)
    only = G.layernorm_bwd(x, dy, m, r, w, want_dx=False, with_bias=False)
    assert only["x"] is None and only["bias"] is None and torch.equal(only["weight"], full["weight"])
    only = G.layernorm_bwd(x, dy, m, r, None, want_dx=False)
    assert only["weight"] is None and torch.equal(only["bias"], full["bias"])


def test_no_rows(G):
    import torch
    x, w = torch.empty((0, 64), device="cuda"), torch.ones(64, device="cuda")
    y, m, r = G.layernorm_fwd(x, w)
    assert y.shape == (0, 64)
    d = G.layernorm_bwd(x, x, m, r, w)
    assert d["x"].shape == (0, 64) and torch.equal(d["weight"], torch.zeros_like(w)) and torch.equal(d["bias"], torch.zeros_like(w))


def test_offsets_past_32_bits(G):
    """Rows behind element 2^31 (and byte 2^32): the last rows equal the same rows alone."""
    import torch
    rows, D = (1 << 31) // 4096 + 5, 4096
    x = torch.empty((rows, D), dtype=torch.bfloat16, device="cuda")
    x[-8:] = torch.randn((8, D), device="cuda").bfloat16()
    x[:-8] = 1.0
    y, m, r = G.layernorm_fwd(x)
    y8, m8, r8 = G.layernorm_fwd(x[-8:].contiguous())
    assert torch.equal(y[-8:], y8) and torch.equal(m[-8:], m8) and torch.equal(r[-8:], r8)
    d = G.layernorm_bwd(x, x, m, r, want_dx=True)
    assert torch.equal(d["x"][-8:], G.layernorm_bwd(x[-8:].contiguous(), x[-8:].contiguous(), m8, r8)["x"])
