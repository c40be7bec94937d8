"""The scan's kernels at training sizes, against the fp64 definition: blocks of 32 and of 16 channels, alone
and in clusters, over many turns (stages, exchange buffers and their phases used again), padded
batches that end in different turns.  Tolerances as in test_gpu_scan.py."""
import pytest

from test_gpu_scan import Case, G, _check

pytestmark = pytest.mark.gpu


def _plan(B, T, D, vec, sms):
    """(channels of a block, blocks of a cluster, turns) forward and backward, by the dispatch's rule."""
    wide = -(-D // 32)
    ch = 16 if D <= 16 or wide * B * 8 <= sms else 32
    tiles, plans = -(-D // ch) * B, []
    for elems in (32 if vec else 16, 16):
        v = 4 if vec else 1
        tok = 8 * (32 // (ch // v)) * (elems // v)
        n = 1
        while n < 16 and tiles * n * 2 <= 2 * sms and n * tok < T:
            n *= 2
        plans.append((ch, n, -(-T // (n * tok))))
    return plans


@pytest.mark.parametrize("B,T,D,lengths,plans", [
    (4, 1500, 2048, None, [(32, 1, 6), (32, 1, 12)]),
    (4, 1500, 2048, [1500, 0, 257, 1281], [(32, 1, 6), (32, 1, 12)]),
    (2, 5000, 1000, [2049, 5000], [(32, 4, 5), (32, 4, 10)]),
    (1, 11000, 640, None, [(32, 8, 6), (32, 8, 11)]),
    (3, 6000, 333, [6000, 1, 3333], [(32, 8, 6), (32, 8, 6)]),
    (8, 700, 1023, [700, 699, 0, 128, 129, 1, 384, 640], [(32, 1, 6), (32, 1, 6)]),
    (1, 45000, 64, None, [(16, 16, 6), (16, 16, 11)]),
    (2, 30000, 48, [30000, 12345], [(16, 16, 4), (16, 16, 8)]),
    (1, 30000, 61, [29999], [(16, 16, 8), (16, 16, 8)]),
])
@pytest.mark.parametrize("x,g,tied,gate_mode", [("bf16", "f32", False, 1), ("f32", "bf16", True, 0)])
def test_many_turns(G, B, T, D, lengths, plans, x, g, tied, gate_mode):
    import torch
    if torch.cuda.get_device_properties(0).multi_processor_count == 148:
        assert _plan(B, T, D, D % 8 == 0, 148) == plans
    _check(G, Case(B, T, D, x=x, g=g, tied=tied, gate_mode=gate_mode, lengths=lengths))
