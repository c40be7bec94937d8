"""Calls on a stream that is passed and is not the current one: outputs, workspace and tensors that the
caller drops keep their memory until that stream is done, whatever the current stream allocates and
writes meanwhile."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    from recurrent_state_memory_b200 import gdr
    gdr.lib()
    return gdr


def _calls(G):
    """name: (inputs, call of them, bytes of its workspace)."""
    import torch
    gen = torch.Generator("cuda").manual_seed(7)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x, g, h0, dh = r(2, 700, 96), r(2, 700, 96), r(2, 96), r(2, 700, 96)
    ck = G.scan_fwd(x, g, h0, want_ckpt=True)[2]
    y, dy, w = r(3000, 512), r(3000, 512), r(512)
    _, mean, rstd = G.layernorm_fwd(y, w)
    nd = G.norm_desc(3000, 512, y.dtype, dy.dtype)
    z, sc = r(16, 8, 20000), r(16, 8)
    parent = torch.randint(0, 8, (16, 8), generator=gen, device="cuda", dtype=torch.int32)
    return {
        "scan_fwd": ((x, g, h0), lambda x, g, h0, **k: G.scan_fwd(x, g, h0, want_ckpt=True, **k), 0),
        "scan_bwd": ((x, g, ck, dh, h0), lambda *a, **k: list(G.scan_bwd(*a, **k).values()), 0),
        "scan_step": ((x[:, 0].contiguous(), g[:, 0].contiguous(), h0), lambda *a, **k: (G.scan_step(*a, **k),), 0),
        "layernorm_fwd": ((y, w, w), G.layernorm_fwd, 0),
        "layernorm_bwd": ((y, dy, mean, rstd, w), lambda *a, **k: list(G.layernorm_bwd(*a, **k).values()),
                          int(G.lib().gdr_layernorm_bwd_workspace_bytes(nd, 1, 1))),
        "beam_select": ((z, sc), lambda *a, **k: G.beam_select(*a, 8, **k),
                        G.beam_workspace_bytes(G.beam_desc(16, 8, 20000, 8, z.dtype))),
        "state_reorder": ((z.view(128, -1)[:, :5000].contiguous(), parent), lambda *a, **k: (G.state_reorder(*a, **k),), 0),
    }


NAMES = ["scan_fwd", "scan_bwd", "scan_step", "layernorm_fwd", "layernorm_bwd", "beam_select", "state_reorder"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_stays_until_the_stream_is_done(G, name):
    """The stream has about a millisecond of other work first; the current one fills all that it is given
    of the inputs', the outputs' and the workspace's sizes, many times over."""
    import torch
    inputs, call, ws = _calls(G)[name]
    want = [v.clone() for v in call(*(v.clone() for v in inputs))]
    side = torch.cuda.Stream()
    for external in (False, True):
        theirs = [v.clone() for v in inputs]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        stream = torch.cuda.ExternalStream(side.cuda_stream) if external else side
        got = list(call(*theirs, stream=stream))
        if name not in ("scan_step", "state_reorder"):      # outputs that are dropped at once
            call(*theirs, stream=stream)
        del theirs
        sizes = {v.numel() * v.element_size() for v in (*inputs, *want)} | ({ws} if ws else set())
        for _ in range(60):
            junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
            del junk
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_work_queued_on_the_current_stream_is_left_alone(G, name):
    """Tensors that the current stream still has to read, and that the caller has dropped, are not taken
    for a call on another stream."""
    import torch
    inputs, call, ws = _calls(G)[name]
    outs = call(*(v.clone() for v in inputs))
    sizes = sorted({v.numel() * v.element_size() for v in outs} | ({ws} if ws else set()))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    theirs = [v.clone() for v in inputs]
    held = [torch.full((n,), 3, dtype=torch.uint8, device="cuda") for n in sizes]
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(2_000_000)
    copies = [torch.empty_like(v) for v in held]
    for c, v in zip(copies, held):
        c.copy_(v)
    del held, v
    keep = call(*theirs, stream=side)
    torch.cuda.synchronize()
    assert all(bool((c == 3).all()) for c in copies) and keep is not None
