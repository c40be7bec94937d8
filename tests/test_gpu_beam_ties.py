"""Beam selection where candidates of beams outside the list tie with candidates in it, or lie as near as
the fp32 sums' error: the order is the 64-bit one, of equal candidates the lowest k * V + v first."""
import pytest

from test_gpu_beam import G, _check, _dt, _make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("k,m", [(4, 1), (4, 2), (8, 1), (8, 4), (8, 8), (16, 3), (64, 5)])
def test_twins_beyond_the_list(G, k, m, x):
    """K equal beams and fewer candidates out than beams: the first beams have them."""
    for seed in range(8):
        z, s = _make(3, 1, 2000 + seed, x, seed=seed)
        _check(G, z.expand(3, k, z.shape[2]).contiguous(), s.expand(3, k).contiguous(), m)


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("k,m", [(8, 8), (8, 3), (16, 16), (33, 20)])
def test_one_better_beam_and_its_twins(G, k, m, x):
    """One beam takes part of the list; the twins of the rest reach past its end."""
    for seed in range(8):
        z, s = _make(2, 1, 2100 + seed, x, seed=50 + seed)
        z, s = z.expand(2, k, z.shape[2]).contiguous(), s.expand(2, k).contiguous()
        s[:, k // 2] += 0.25
        _check(G, z, s, m)


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("k,m", [(6, 1), (6, 3), (16, 1), (16, 7), (48, 9)])
def test_third_beams_within_the_error(G, k, m, x):
    """Beams of different logits whose best candidates lie within a few 1e-6 of one another, most of
    them behind the list's end."""
    import torch
    for seed in range(8):
        z, _ = _make(1, k, 3000, x, seed=200 + seed, banned=0)
        best = z.double().log_softmax(2).amax(2)
        s = (-10 - best).float()
        s += (torch.randperm(k, device="cuda")[None] % 5 - 2) * 1e-6
        _check(G, z, s, m)


@pytest.mark.parametrize("m", [1, 2, 5])
def test_finished_beams_at_the_lists_end(G, m):
    """A finished beam's exact score between scores of beams that the fp32 sums cannot order."""
    import torch
    for seed in range(8):
        z, _ = _make(1, 8, 4000, "f32", seed=300 + seed, banned=0)
        s = (-10 - z.double().log_softmax(2).amax(2)).float()
        f = torch.zeros((1, 8), dtype=torch.bool, device="cuda")
        f[0, 3] = f[0, 6] = True
        s[f] = -10.0
        _check(G, z, s, m, f, 7)


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_twins_of_large_vocabularies(G, x):
    """Pieces of 2048 and of 8192 elements, several a row."""
    for g, k, v in ((2, 4, 50001), (20, 8, 20011)):
        z, s = _make(g, 1, v, x, seed=9)
        _check(G, z.expand(g, k, v).contiguous(), s.expand(g, k).contiguous(), 2)


@pytest.mark.parametrize("m", [2, 7])
def test_twins_among_masked_and_empty_beams(G, m):
    """Fewer finite candidates than asked for, twins among them; the rest is filled by index."""
    import torch
    z, s = _make(2, 1, 900, "f32", seed=11)
    z, s = z.expand(2, 6, 900).contiguous(), s.expand(2, 6).contiguous()
    z[0, :, 2:] = -float("inf")
    z[1, :, 1:] = -float("inf")
    s[:, 1] = -float("inf")
    z[:, 4] = float("nan")
    _check(G, z, s, m)
