"""Refusals of the scan, the layer norm, the beam selection and the state reorder, before anything
is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from recurrent_state_memory_b200 import build as gdr_build


@pytest.fixture(scope="module")
def G():
    gdr_build.build()
    from recurrent_state_memory_b200 import gdr
    gdr.lib()
    return gdr


P = ctypes.c_void_p(1 << 20)            # never dereferenced: every call below fails its checks first
ODD = ctypes.c_void_p((1 << 20) + 1)
HALF = ctypes.c_void_p((1 << 20) + 2)
FOUR = ctypes.c_void_p((1 << 20) + 4)


def test_exports(G):
    assert {"gdr_scan_fwd", "gdr_scan_bwd", "gdr_scan_step", "gdr_layernorm_fwd", "gdr_layernorm_bwd",
            "gdr_layernorm_bwd_workspace_bytes", "gdr_beam_select", "gdr_beam_select_workspace_bytes",
            "gdr_state_reorder"} <= set(G.header_symbols())
    assert G.status_string(8) == "GDR_ERR_INDEX" and G.lib().gdr_abi_version() == 6


def test_scan_refusals(G):
    L = G.lib()

    def desc(B=2, T=10, D=8, x_row=0, g_row=0, **kw):
        d = G.scan_desc(B, T, D, torch.bfloat16, torch.float32, torch.bfloat16, x_row=x_row, g_row=g_row)
        for k, v in kw.items():
            setattr(d, k, v)
        return d

    fwd = lambda d, x=P, g=P, h0=P, n=None, h=P, hT=P, ck=P: L.gdr_scan_fwd(d, x, g, h0, n, h, hT, ck, None)
    bwd = lambda d, x=P, g=P, ck=P, dx=P, dg=P, dh=P: L.gdr_scan_bwd(d, x, g, ck, None, dh, None, dx, dg, None, None)
    step = lambda d, x=P, g=P, h=P, o=P: L.gdr_scan_step(d, x, g, h, o, None)
    for call in (fwd, bwd, step):
        assert call(None) == G.GDR_ERR_INVALID_ARG
        for bad in (dict(B=-1), dict(T=-1), dict(D=-1), dict(x_dtype=2), dict(g_dtype=-1), dict(out_dtype=7),
                    dict(gate_mode=2), dict(tied=2), dict(x_row=7), dict(g_row=-8)):
            assert call(desc(**bad)) == G.GDR_ERR_INVALID_ARG, bad
        assert call(desc(), x=None) == G.GDR_ERR_INVALID_ARG
        assert call(desc(), g=None) == G.GDR_ERR_INVALID_ARG
        assert call(desc(), x=ODD) == G.GDR_ERR_INVALID_ARG         # not its element's alignment
        assert call(desc(), g=HALF) == G.GDR_ERR_INVALID_ARG
        assert call(desc(B=0)) == G.GDR_OK and call(desc(D=0), x=None) == G.GDR_OK
    assert fwd(desc(), h=None) == G.GDR_ERR_INVALID_ARG
    assert fwd(desc(), h0=HALF) == G.GDR_ERR_INVALID_ARG and fwd(desc(), hT=HALF) == G.GDR_ERR_INVALID_ARG
    assert fwd(desc(), h=FOUR) == G.GDR_ERR_INVALID_ARG and fwd(desc(), ck=FOUR) == G.GDR_ERR_INVALID_ARG
    assert fwd(desc(), n=HALF) == G.GDR_ERR_INVALID_ARG
    assert fwd(desc(T=0), x=None, g=None, h=None, h0=None, hT=None) == G.GDR_OK
    for missing in ("ck", "dx", "dg"):
        assert bwd(desc(), **{missing: None}) == G.GDR_ERR_INVALID_ARG
        assert bwd(desc(), **{missing: HALF}) == G.GDR_ERR_INVALID_ARG
    for bad in (dict(B=1 << 27), dict(T=(1 << 30) + 1), dict(D=65535 * 16 + 1)):
        assert fwd(desc(**bad)) == G.GDR_ERR_UNSUPPORTED and bwd(desc(**bad)) == G.GDR_ERR_UNSUPPORTED
    assert step(desc(), h=None) == G.GDR_ERR_INVALID_ARG
    assert step(desc(), o=ODD) == G.GDR_ERR_INVALID_ARG and step(desc(), h=HALF) == G.GDR_ERR_INVALID_ARG
    assert bwd(desc(), dh=ODD) == G.GDR_ERR_INVALID_ARG


def test_layernorm_refusals(G):
    L = G.lib()

    def desc(**kw):
        d = G.norm_desc(4, 64, torch.bfloat16, torch.bfloat16)
        for k, v in kw.items():
            setattr(d, k, v)
        return d

    fwd = lambda d, x=P, y=P, w=P: L.gdr_layernorm_fwd(d, x, w, P, y, P, P, None)
    bwd = lambda d, x=P, dy=P, mean=P, ws=P, n=1 << 30, dx=P: L.gdr_layernorm_bwd(d, x, dy, P, mean, P, dx, P, P, ws, n, None)
    for call in (fwd, bwd):
        assert call(None) == G.GDR_ERR_INVALID_ARG
        for bad in (dict(rows=-1), dict(x_dtype=3), dict(y_dtype=-1), dict(w_dtype=2), dict(eps=-1.0),
                    dict(eps=float("nan"))):
            assert call(desc(**bad)) == G.GDR_ERR_INVALID_ARG, bad
        assert call(desc(D=0)) == G.GDR_ERR_UNSUPPORTED and call(desc(D=(1 << 20) + 1)) == G.GDR_ERR_UNSUPPORTED
        assert call(desc(rows=(1 << 40) + 1)) == G.GDR_ERR_UNSUPPORTED
        assert call(desc(), x=None) == G.GDR_ERR_INVALID_ARG
        assert call(desc(), x=ODD) == G.GDR_ERR_INVALID_ARG
    assert fwd(desc(), y=None) == G.GDR_ERR_INVALID_ARG and fwd(desc(), w=HALF) == G.GDR_ERR_INVALID_ARG
    assert bwd(desc(), dy=None) == G.GDR_ERR_INVALID_ARG and bwd(desc(), mean=None) == G.GDR_ERR_INVALID_ARG
    need = lambda d, w, b: L.gdr_layernorm_bwd_workspace_bytes(d, w, b)
    assert need(desc(), 0, 0) == 0 and need(desc(D=0), 1, 1) == 0
    assert need(desc(), 1, 1) == 2 * need(desc(), 1, 0) > 0
    assert bwd(desc(), ws=None) == G.GDR_ERR_WORKSPACE
    assert bwd(desc(), ws=FOUR) == G.GDR_ERR_INVALID_ARG and bwd(desc(), mean=HALF) == G.GDR_ERR_INVALID_ARG
    assert bwd(desc(), n=need(desc(), 1, 1) - 1) == G.GDR_ERR_WORKSPACE


def test_beam_refusals(G):
    L = G.lib()

    def desc(**kw):
        d = G.beam_desc(2, 4, 100, 8, torch.float32)
        for k, v in kw.items():
            setattr(d, k, v)
        return d

    def call(d, z=P, s=P, f=None, o=P, p=P, t=P, ws=P, n=1 << 30):
        return L.gdr_beam_select(d, z, s, f, o, p, t, ws, n, None)

    assert call(None) == G.GDR_ERR_INVALID_ARG
    for bad in (dict(G=-1), dict(V=0), dict(row=99), dict(x_dtype=5), dict(V=2, K=3, M=7)):
        assert call(desc(**bad)) == G.GDR_ERR_INVALID_ARG, bad
    for bad in (dict(K=0), dict(K=65), dict(M=0), dict(M=65), dict(V=1 << 29), dict(G=1 << 30)):
        assert call(desc(**bad)) == G.GDR_ERR_UNSUPPORTED, bad
        assert L.gdr_beam_select_workspace_bytes(desc(**bad)) == 0
    for eos in (-1, 100):
        assert call(desc(eos=eos), f=P) == G.GDR_ERR_INVALID_ARG
    for name in "zsopt":
        assert call(desc(), **{name: None}) == G.GDR_ERR_INVALID_ARG
        assert call(desc(), **{name: HALF}) == G.GDR_ERR_INVALID_ARG
    assert call(desc(), ws=None) == G.GDR_ERR_WORKSPACE
    need = L.gdr_beam_select_workspace_bytes(desc())
    assert need > 0 and call(desc(), n=need - 1) == G.GDR_ERR_WORKSPACE
    assert call(desc(G=0)) == G.GDR_OK


def test_reorder_refusals(G):
    L = G.lib()
    call = lambda L_=1, g=2, k=4, n=64, S=P, p=P: L.gdr_state_reorder(G.ReorderDesc(L_, g, k, n), S, p, None)
    assert L.gdr_state_reorder(None, P, P, None) == G.GDR_ERR_INVALID_ARG
    assert call(L_=-1) == G.GDR_ERR_INVALID_ARG and call(g=-1) == G.GDR_ERR_INVALID_ARG
    assert call(k=0) == G.GDR_ERR_UNSUPPORTED and call(k=65) == G.GDR_ERR_UNSUPPORTED
    assert call(L_=1 << 16, g=1 << 16) == G.GDR_ERR_UNSUPPORTED
    assert call(S=None) == G.GDR_ERR_INVALID_ARG and call(p=None) == G.GDR_ERR_INVALID_ARG
    assert call(p=HALF) == G.GDR_ERR_INVALID_ARG
    assert call(n=0) == G.GDR_OK and call(L_=0, S=None) == G.GDR_OK and call(g=0) == G.GDR_OK


def test_binding_refuses_what_is_not_on_the_gpu(G):
    x = torch.zeros(2, 3, 4)
    for call in (lambda: G.scan_fwd(x, x), lambda: G.scan_step(x[0], x[0], x[0]), lambda: G.layernorm_fwd(x),
                 lambda: G.beam_select(x, x[..., 0]), lambda: G.state_reorder(x, torch.zeros(1, 2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_takes_row_slices_only(G):
    wide, row_stride = torch.zeros(2, 5, 12), G._ops().row_stride
    assert row_stride(wide, "x") == 0
    assert row_stride(wide[..., 4:8], "x") == 12
    assert row_stride(wide[:1, :, :8], "x") == 12
    for bad in (wide[:, ::2], wide[:, :4, :8], wide[..., ::2], wide.transpose(1, 2), wide[0].expand(2, 5, 12)):
        with pytest.raises(ValueError, match="contiguous"):
            row_stride(bad, "x")
