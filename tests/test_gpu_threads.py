"""Host threads that call the library at once, each on a stream of its own: no call fails, and the results
are the single thread's."""
import threading

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    from recurrent_state_memory_b200 import gdr
    gdr.lib()
    return gdr


def _p(t):
    import ctypes
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def test_the_first_call_of_a_host_thread(G):
    """A thread that has made no other CUDA call, after the library has been used on another one: the scan
    and the tensor-core forward, whose tensor maps need the thread's context."""
    import torch
    L, B, T, D = G.lib(), 2, 300, 64
    x, g = torch.randn(2, B, T, D, device="cuda").bfloat16()
    ref, h = G.scan_fwd(x, g)[0], torch.empty_like(x)
    scan = G.scan_desc(B, T, D, x.dtype, g.dtype, h.dtype)
    q, k, v = torch.nn.functional.normalize(torch.randn(3, 1, 128, 2, 128, device="cuda"), dim=-1).bfloat16()
    beta = torch.full((1, 128, 2), 0.5, device="cuda")
    a = torch.randn(1, 128, 2, 128, device="cuda")
    want, got = G.chunk_fwd(q, k, v, a, beta, algo="tcgen05_split", want_state=False)[0], torch.empty_like(v)
    fwd = G.fwd_desc(1, 2, 128, 128, 128, q.dtype, got.dtype, algo="tcgen05_split")
    n = G.workspace_bytes(fwd)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    calls = [lambda: L.gdr_scan_fwd(scan, _p(x), _p(g), None, None, _p(h), None, None, None),
             lambda: L.gdr_chunk_fwd(fwd, _p(q), _p(k), _p(v), _p(a), _p(beta), None, None, _p(got), None, _p(ws), n, None)]
    for call in calls:
        out = []
        t = threading.Thread(target=lambda: out.append((call(), L.gdr_last_error_detail())))
        t.start()
        t.join()
        assert out == [(G.GDR_OK, b"")]
    torch.cuda.synchronize()
    assert torch.equal(h, ref) and torch.equal(got, want)
