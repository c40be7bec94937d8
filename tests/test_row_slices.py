"""Row slices that the scan and the beam selection take as they are: a dimension of one has no say."""
import pytest
import torch

from recurrent_state_memory_b200 import build, gdr


@pytest.fixture(scope="module")
def row_stride():
    build.build()
    return gdr._ops().row_stride


def test_dimensions_of_one(row_stride):
    wide = torch.zeros(3, 12)
    assert row_stride(wide[:, :8].unsqueeze(1), "x") == 12             # one token of 3 sequences
    assert row_stride(torch.zeros(3, 7, 10)[:, -1:], "x") == 70         # the last token's logits
    assert row_stride(torch.zeros(3, 7, 10)[:, -1:, 2:9], "x") == 70
    assert row_stride(torch.zeros(3, 5, 10)[..., 4:5], "x") == 10       # one channel
    assert row_stride(torch.zeros(3, 1, 10)[..., :4], "x") == 10
    assert row_stride(torch.zeros(1, 5, 10)[..., :4], "x") == 10
    assert row_stride(torch.zeros(6, 4).t()[:1].t().unsqueeze(0), "x") == 4
    assert row_stride(torch.zeros(4, 1, 1, 9)[..., :3], "x") == 9


def test_still_refused(row_stride):
    wide = torch.zeros(2, 5, 12)
    for bad in (wide[:, ::2], wide[:, :4, :8], wide[..., ::2], wide.transpose(1, 2), wide[0].expand(2, 5, 12),
                wide[:, :1, :8].expand(2, 5, 8), torch.zeros(12).as_strided((5, 4), (2, 1)),
                torch.zeros(1).expand(3, 4), torch.zeros(4, 1).expand(4, 3)):
        with pytest.raises(ValueError, match="contiguous"):
            row_stride(bad, "x")


@pytest.mark.gpu
def test_the_calls_take_them():
    gen = torch.Generator("cuda").manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    wide, g = r(5, 24), r(5, 9, 16)
    x = wide[:, :16].unsqueeze(1)
    a = gdr.scan_fwd(x, g[:, 4:5], want_ckpt=True)
    b = gdr.scan_fwd(x.contiguous(), g[:, 4:5].contiguous(), want_ckpt=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    d, e = gdr.scan_bwd(x, g[:, 4:5], a[2], x.contiguous()), gdr.scan_bwd(x.contiguous(), g[:, 4:5].contiguous(), b[2], x.contiguous())
    assert all(torch.equal(d[k], e[k]) for k in d)
    y = r(5, 9, 16)
    one = gdr.scan_fwd(y[..., 3:4], y[..., 4:5])
    assert torch.equal(one[0], gdr.scan_fwd(y[..., 3:4].contiguous(), y[..., 4:5].contiguous())[0])
    logits, s = r(6, 7, 501), r(6, 1)
    assert all(torch.equal(p, q) for p, q in zip(gdr.beam_select(logits[:, -1:], s, 5), gdr.beam_select(logits[:, -1:].contiguous(), s, 5)))
