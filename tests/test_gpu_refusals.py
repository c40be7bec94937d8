"""Arguments of the scan, layer norm and beam calls that are refused before anything is allocated or launched."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    from recurrent_state_memory_b200 import gdr
    gdr.lib()
    return gdr


def test_a_workspace_that_is_less_memory_than_its_size(G):
    """Expanded and strided tensors have other memory than numel * element_size bytes from their start on."""
    import torch
    x = torch.randn(64, 256, device="cuda")
    _, mean, rstd = G.layernorm_fwd(x)
    z, s = torch.randn(2, 4, 3000, device="cuda"), torch.randn(2, 4, device="cuda")
    for ws in (torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 24),
               torch.empty(1 << 20, 64, dtype=torch.uint8, device="cuda")[:, ::2]):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            G.layernorm_bwd(x, x, mean, rstd, workspace=ws)
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            G.beam_select(z, s, workspace=ws)
    for ws in (torch.empty(1 << 24, dtype=torch.uint8), torch.empty(16, dtype=torch.uint8, device="cuda")):
        with pytest.raises(ValueError if not ws.is_cuda else G.GdrError):
            G.layernorm_bwd(x, x, mean, rstd, workspace=ws)
        with pytest.raises(ValueError if not ws.is_cuda else G.GdrError):
            G.beam_select(z, s, workspace=ws)


def test_more_candidates_than_there_may_be(G):
    """Refused by the library's own error, without memory for as many outputs."""
    import torch
    z, s = torch.randn(64, 4, 300, device="cuda"), torch.randn(64, 4, device="cuda")
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    for n in (0, -3, 65, 1 << 30):
        with pytest.raises(G.GdrError, match="1 .. 64"):
            G.beam_select(z, s, n)
    assert torch.cuda.max_memory_allocated() == before
    assert [t.shape for t in G.beam_select(z[:0], s[:0], 3)] == [(0, 3)] * 3
