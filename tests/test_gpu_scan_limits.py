"""The scan at sizes past 32 bits."""
import pytest

pytestmark = pytest.mark.gpu


def test_more_than_2_to_the_33_tokens():
    """8200 sequences of 2^20 tokens, one channel (69 GB): the same as the last and the first sequences alone."""
    import torch
    from recurrent_state_memory_b200 import gdr as G
    B, T = 8200, 1 << 20
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("90 GB of free memory are needed")
    gen = torch.Generator("cuda").manual_seed(4)
    x = torch.empty((B, T, 1), dtype=torch.bfloat16, device="cuda")
    g = torch.empty((B, T, 1), device="cuda")
    for at in range(0, B, 410):
        x[at:at + 410] = torch.randn((410, T, 1), generator=gen, device="cuda")
        g[at:at + 410].normal_(generator=gen)
    h, h_T = G.scan_fwd(x, g)
    for part in (slice(0, 3), slice(B // 2, B // 2 + 2), slice(B - 10, B)):
        a, b = G.scan_fwd(x[part].contiguous(), g[part].contiguous())
        scale = a.abs().max().float()
        assert (a.float() - h[part].float()).abs().max() <= 2 ** -7 * scale     # other clusters, one rounding
        assert (b - h_T[part]).abs().max() <= 1e-5 * scale
    assert G.query_device_status() == G.GDR_OK
    del x, g, h, h_T, a, b
    torch.cuda.empty_cache()
