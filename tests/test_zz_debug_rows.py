"""The debug build's index checks in the layer norm's rows of every kind (shifted by few lanes, by warps and
by blocks, one by one, wide, read again), at the tensor's two ends, and in the beam lists that overflow."""
import pytest

from test_zz_debug_block import G, _both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x,y", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,D", [(1, 9), (300, 9), (41, 14), (1, 333), (37, 333), (19, 129), (21, 2047), (11, 5001),
                                    (7, 8190), (3, 10240), (5, 16384), (2, 17001)])
def test_layernorm(G, rows, D, x, y):
    import torch
    t = {"bf16": torch.bfloat16, "f32": torch.float32}
    gen = torch.Generator("cuda").manual_seed(rows + D)
    a, dy = torch.randn(rows, D, generator=gen, device="cuda").to(t[x]), torch.randn(rows, D, generator=gen, device="cuda").to(t[y])
    w = torch.randn(D, generator=gen, device="cuda")

    def run(gdr):
        out, m, r = gdr.layernorm_fwd(a, w, w, out_dtype=t[y])
        d = gdr.layernorm_bwd(a, dy, m, r, w)
        return out, m, r, d["x"], d["weight"], d["bias"]

    _both(G, run)


@pytest.mark.parametrize("g,k,v", [(1, 2, 5000), (40, 8, 9001)])
def test_beam_lists_that_overflow(G, g, k, v):
    import torch
    z, s = torch.zeros(g, k, v, device="cuda"), torch.zeros(g, k, device="cuda")
    _both(G, lambda gdr: gdr.beam_select(z, s, 16))


@pytest.mark.parametrize("B,T,D", [(2, 2000, 333), (4, 1500, 2048), (3, 700, 1023)])
def test_scan_in_blocks_of_32_channels(G, B, T, D):
    import torch
    gen = torch.Generator("cuda").manual_seed(T + D)
    x, g, dh = torch.randn(3, B, T, D, generator=gen, device="cuda").bfloat16()
    n = torch.tensor([T, T // 2 + 1, 0, 70][:B], dtype=torch.int32, device="cuda")

    def run(gdr):
        h, hT, ck = gdr.scan_fwd(x, g, lengths=n, want_ckpt=True)
        d = gdr.scan_bwd(x, g, ck, dh, hT, lengths=n)
        return h, hT, ck, d["x"], d["g"], d["h0"]

    _both(G, run)
