"""Beam selection at the ends of its documented range: as many beams as G * K < 2^31 allows."""
import pytest

pytestmark = pytest.mark.gpu


def test_beams_up_to_the_limit():
    """2^31 - 64 beams of one token each (47 GB): the grid's last rows lie past 2^31.  Every group's best is the
    largest score, of equal ones the first."""
    import torch
    from recurrent_state_memory_b200 import gdr as G
    k, g = 64, (1 << 25) - 1
    if torch.cuda.mem_get_info()[0] < 70 << 30:
        pytest.skip("70 GB of free memory are needed")
    z = torch.zeros((g, k, 1), dtype=torch.bfloat16, device="cuda")
    s = torch.rand((g, k), generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    best, parent, token = G.beam_select(z, s, 1)
    del z
    lane = torch.arange(k, dtype=torch.int32, device="cuda")
    for at in range(0, g, 1 << 22):
        part = s[at:at + (1 << 22)]
        top = part.amax(1, keepdim=True)
        first = torch.where(part == top, lane, k).amin(1, keepdim=True)
        assert torch.equal(best[at:at + (1 << 22)], top)
        assert torch.equal(parent[at:at + (1 << 22)], first.int())
    assert not bool(token.any())
    assert G.query_device_status() == G.GDR_OK
    del s, best, parent, token, part, top, first
    torch.cuda.empty_cache()
