"""Beam selection of ordinary batches, whose rows are cut into pieces of 8192 elements (32 a thread), against
the fp64 definition: full and last pieces, 16-byte and single loads, both types, ties, masks, lists
that overflow, as many candidates as there may be."""
import pytest

from test_gpu_beam import G, _check, _dt, _make

pytestmark = pytest.mark.gpu
VS = [8191, 8192, 8193, 20011, 32000]


def _size(v):
    """Groups of 8 beams: enough rows that the pieces are large ones."""
    pieces = -(-v // 8192)
    g = -(-2 * 148 // (8 * pieces))
    assert g * 8 * pieces >= 296
    return g, 8


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("v", VS)
@pytest.mark.parametrize("m", [1, 8, 64])
def test_vocabularies(G, x, v, m):
    g, k = _size(v)
    _check(G, *_make(g, k, v, x, seed=m), m)


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("v", [8193, 32000])
def test_rows_that_start_on_no_16_bytes(G, x, v):
    """Slices of wider rows (NaN behind them), and logits that start inside 16 bytes."""
    import torch
    g, k = _size(v)
    z, s = _make(g, k, v, x, seed=21)
    wide = torch.full((g, k, v + 3), float("nan"), device="cuda", dtype=z.dtype)
    wide[..., :v] = z
    _check(G, wide[..., :v], s, 8)
    flat = torch.empty(z.numel() + 1, dtype=z.dtype, device="cuda")
    flat[1:] = z.reshape(-1)
    _check(G, flat[1:].view(g, k, v), s, 8)


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("v", [8192, 20011])
@pytest.mark.parametrize("m", [3, 40])
def test_everything_is_equal(G, x, v, m):
    """Every element of every piece reaches the mark."""
    import torch
    g, k = _size(v)
    _check(G, torch.zeros((g, k, v), device="cuda", dtype=_dt(x)), torch.full((g, k), -3.0, device="cuda"), m)


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_few_values_and_many_ties(G, x):
    import torch
    g, k = _size(20011)
    gen = torch.Generator("cuda").manual_seed(5)
    z = torch.randint(-4, 5, (g, k, 20011), generator=gen, device="cuda").to(_dt(x))
    _check(G, z, torch.randint(-2, 1, (g, k), generator=gen, device="cuda").float(), 48)


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("v", [8193, 32000])
def test_masks_and_poisons(G, x, v):
    """Mostly masked rows, rows of one token, of none, of lowest values; NaN, +inf; scores of -inf and NaN;
    finished beams."""
    import torch
    g, k = _size(v)
    z, s = _make(g, k, v, x, seed=31, banned=0)
    gen = torch.Generator("cuda").manual_seed(6)
    z[torch.rand(z.shape, generator=gen, device="cuda") < 0.999] = -float("inf")
    z[0] = -float("inf")
    z[1, 0] = -float("inf")
    z[1, 0, v - 1] = 1.0
    z[1, 1] = torch.finfo(z.dtype).min
    z[1, 2, 17] = float("nan")
    z[1, 3, v - 1] = float("inf")
    s[1, 4] = -float("inf")
    s[1, 5] = float("nan")
    f = torch.zeros((g, k), dtype=torch.bool, device="cuda")
    f[2:, ::3] = True
    _check(G, z, s, 8, f, 2)
    _check(G, z, s, 64, f, v - 1)


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_descending_rows(G, x):
    """The best of a row lie side by side in few lanes."""
    import torch
    g, k = _size(32000)
    z = torch.linspace(9, -9, 32000, device="cuda").expand(g, k, 32000).contiguous().to(_dt(x))
    s = -torch.rand((g, k), generator=torch.Generator("cuda").manual_seed(8), device="cuda")
    _check(G, z, s, 20)
