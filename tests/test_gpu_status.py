"""The device status word: what kernels of different files leave there arrives in one query, once."""
import pytest

pytestmark = pytest.mark.gpu


def test_every_kernels_report_arrives_once():
    import torch
    from recurrent_state_memory_b200 import gdr as G
    assert G.query_device_status() == G.GDR_OK
    S, bad = torch.zeros(4, 8, device="cuda"), torch.full((1, 4), 9, dtype=torch.int32, device="cuda")
    # log-decays that leave the tensor-core form's range (the forward of gdr.cu), then a bad parent (beam.cu)
    q = torch.randn(1, 128, 1, 128, device="cuda").bfloat16()
    g = torch.full((1, 128, 1, 128), -200.0, device="cuda")
    beta = torch.full((1, 128, 1), 0.5, device="cuda")
    fwd = lambda: G.chunk_fwd(q, q, q, g, beta, gate_mode=G.GATE_LOGDECAY, algo="tcgen05", qk_l2norm=True)
    fwd()
    alone = G.query_device_status()
    fwd()
    side = torch.cuda.Stream()
    G.state_reorder(S, bad, stream=side)
    torch.cuda.synchronize()
    both = G.query_device_status(side)
    assert both == G.GDR_ERR_INDEX and alone in (G.GDR_OK, G.GDR_ERR_RANGE)
    assert G.query_device_status() == G.GDR_OK                 # the forward's report went with it
    G.state_reorder(S, bad)
    assert G.query_device_status() == G.GDR_ERR_INDEX and G.query_device_status() == G.GDR_OK
