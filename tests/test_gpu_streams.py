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
    q, k, v, rk = (torch.nn.functional.normalize(r(2, 512, 4, 128), dim=-1).bfloat16() for _ in range(4))
    a, beta, S = r(2, 512, 4, 128), torch.rand((2, 512, 4), generator=gen, device="cuda"), r(2, 4, 128, 128) * 0.1
    fd = G.fwd_desc(2, 4, 512, 128, 128, q.dtype, q.dtype)
    rv, zr, gr = r(2, 512, 4, 128).bfloat16(), r(2, 512, 4, 64), r(2, 512, 4)
    parent = torch.randint(0, 8, (16, 8), generator=gen, device="cuda", dtype=torch.int32)
    return {
        "chunk_fwd": ((q, k, v, a, beta), G.chunk_fwd, G.workspace_bytes(fd)),
        "chunk_bwd": ((q, k, v, a, beta, S, v), lambda *a, **k: [t for t in G.chunk_bwd(*a, **k).values() if t is not None],
                      G.bwd_workspace_bytes(fd)),
        "decode_step": ((q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(), a[:, 0].contiguous(),
                         beta[:, 0].contiguous(), S), lambda *a, **k: (G.decode_step(*a, **k),), 0),
        "raven_fwd": ((rk, k, rv, zr, gr), lambda *a, **k: G.raven_fwd(*a, topk=8, **k),
                      G.raven_workspace_bytes(G.raven_desc(2, 4, 512, 128, 8))),
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


NAMES = ["chunk_fwd", "chunk_bwd", "decode_step", "raven_fwd", "scan_fwd", "scan_bwd", "scan_step", "layernorm_fwd",
         "layernorm_bwd", "beam_select", "state_reorder"]


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
        if name not in ("scan_step", "state_reorder", "decode_step"):      # outputs that are dropped at once
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


@pytest.mark.parametrize("name", NAMES)
def test_the_default_stream_from_another_one(G, name):
    """The passed stream is the default one and the current stream is not."""
    import torch
    inputs, call, _ = _calls(G)[name]
    want = [v.clone() for v in call(*(v.clone() for v in inputs))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        theirs = [v.clone() for v in inputs]
        torch.cuda.default_stream().wait_stream(side)
        got = call(*theirs, stream=torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", [n for n in NAMES if n not in ("scan_step", "state_reorder", "decode_step")])
def test_captured_on_a_branch(G, name):
    """A graph whose call runs on a stream that branches off the captured one; the graph's memory is its own
    and replays give the same again."""
    import torch
    inputs, call, _ = _calls(G)[name]
    want = [v.clone() for v in call(*inputs)]
    side = torch.cuda.Stream()
    call(*inputs, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = list(call(*inputs, stream=side))
        call(*inputs, stream=side)                      # its outputs go at once
        torch.cuda.current_stream().wait_stream(side)
        sums = [v.double().sum() for v in got]
    for _ in range(3):
        junk = [torch.full_like(v, 7) for v in got]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(sums) == len(got)
        del junk
    del got, sums
    torch.cuda.synchronize()
    assert [torch.equal(a, b) for a, b in zip(call(*inputs), want)] == [True] * len(want)
