"""The debug build's index checks in the scan, the layer norm, the beam selection and the state
reorder: on ragged shapes through every variant (vector and one-element rows, clusters, two groups a
block, blocks and lane groups) no check fails and the results are the default build's."""
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    from recurrent_state_memory_b200 import build, gdr
    default = gdr.LIB_PATH
    if not os.path.exists(build.LIB_DEBUG):
        pytest.fail("libgdr_debug.so is missing: __graft_entry__.build() builds it")
    yield gdr, default, build.LIB_DEBUG
    gdr.use_library(default)


def _both(G, run):
    """run() on both builds: the debug build's checks hold; the results, of the compiler's own
    contractions alone, are near each other."""
    import torch
    gdr, default, dbg = G
    res = []
    for path in (default, dbg):
        gdr.use_library(path)
        out = [x.clone() for x in run(gdr) if x is not None]
        torch.cuda.synchronize()
        assert gdr.query_device_status() == gdr.GDR_OK
        if path == dbg:
            assert gdr.debug_bounds_site() == 0
        res.append(out)
    for a, b in zip(*res):
        if a.dtype in (torch.int32, torch.uint8):
            assert torch.equal(a, b)
        else:
            scale = a.double().abs().max().clamp_min(1e-30)
            assert ((a.double() - b.double()).abs().max() / scale) <= (8e-3 if a.dtype == torch.bfloat16 else 1e-5)


@pytest.mark.parametrize("B,T,D", [(2, 300, 64), (3, 777, 61), (1, 5000, 16), (1, 5000, 3), (2, 1, 7), (40, 130, 256)])
def test_scan(G, B, T, D):
    import torch
    gen = torch.Generator("cuda").manual_seed(T + D)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x, g, h0, dh = r(B, T, D).bfloat16(), r(B, T, D), r(B, D), r(B, T, D).bfloat16()
    n = torch.randint(0, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)

    def run(gdr):
        h, hT, ck = gdr.scan_fwd(x, g, h0, tied=True, lengths=n, want_ckpt=True)
        d = gdr.scan_bwd(x, g, ck, dh, h0, tied=True, lengths=n)
        s = h0.clone()
        return h, hT, ck, d["x"], d["g"], d["h0"], gdr.scan_step(x[:, 0], g[:, 0], s), s

    _both(G, run)


@pytest.mark.parametrize("rows,D", [(33, 5), (1000, 128), (17, 250), (9, 1030), (40, 4096), (3, 9000), (2, 20001)])
def test_layernorm(G, rows, D):
    import torch
    gen = torch.Generator("cuda").manual_seed(rows + D)
    x, dy = torch.randn(2, rows, D, generator=gen, device="cuda").bfloat16()
    w = torch.randn(D, generator=gen, device="cuda")

    def run(gdr):
        y, m, r = gdr.layernorm_fwd(x, w, w)
        d = gdr.layernorm_bwd(x, dy, m, r, w)
        return y, m, r, d["x"], d["weight"], d["bias"]

    _both(G, run)


@pytest.mark.parametrize("g,k,v,m", [(2, 4, 1000, 8), (1, 3, 20011, 64), (3, 64, 300, 5), (40, 8, 9001, 8)])
def test_beam_and_reorder(G, g, k, v, m):
    import torch
    gen = torch.Generator("cuda").manual_seed(v)
    z = torch.randn(g, k, v, generator=gen, device="cuda") * 3
    s = torch.randn(g, k, generator=gen, device="cuda")
    S0 = torch.randn(2, g * k, 37, generator=gen, device="cuda")

    def run(gdr):
        sc, p, t = gdr.beam_select(z, s, m)
        S = S0.clone()
        if m >= k:
            gdr.state_reorder(S, p[:, :k].contiguous(), layers=True)
        return sc, p, t, S

    _both(G, run)
