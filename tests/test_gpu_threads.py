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


def _at_once(L, calls, rounds):
    """Every call (C entries through ctypes, which leave Python's lock) in a thread of its own, over and
    over: what went wrong."""
    wrong, go = set(), threading.Barrier(len(calls))

    def work(call):
        go.wait()
        for _ in range(rounds):
            if call() != 0:
                wrong.add(L.gdr_last_error_detail().decode())

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return wrong


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


def test_scan_with_different_clusters(G):
    """The same kernel in clusters of 16 and alone."""
    import torch
    L, held, calls, ref = G.lib(), [], [], []
    for B, T in ((1, 8000), (90, 40), (90, 40)):
        D = 64
        x, g = torch.randn(2, B, T, D, device="cuda").bfloat16()
        ref.append(G.scan_fwd(x, g, want_ckpt=True))
        h, ck = torch.empty_like(x), torch.empty_like(ref[-1][2])
        desc, st = G.scan_desc(B, T, D, x.dtype, g.dtype, h.dtype), torch.cuda.Stream()
        held.append((x, g, h, ck, desc, st))
        calls.append(lambda d=desc, a=x, b=g, o=h, c=ck, s=st: L.gdr_scan_fwd(
            d, _p(a), _p(b), None, None, _p(o), None, _p(c), s.cuda_stream))
    torch.cuda.synchronize()
    assert _at_once(L, calls, 3000) == set()
    torch.cuda.synchronize()
    for r, v in zip(ref, held):
        assert torch.equal(r[0], v[2]) and torch.equal(r[2], v[3])


def test_wide_norm_with_and_without_sums(G):
    """The same kernel with shared memory for the sums and without any."""
    import torch
    L, rows, D = G.lib(), 5, 16384
    x, dy = torch.randn(2, rows, D, device="cuda").bfloat16()
    _, mean, rstd = G.layernorm_fwd(x)
    ref = G.layernorm_bwd(x, dy, mean, rstd)
    desc = G.norm_desc(rows, D, x.dtype, dy.dtype)
    held, calls = [], []
    for sums in (True, False, False, True):
        dx, st = torch.empty_like(x), torch.cuda.Stream()
        db = torch.empty(D, device="cuda") if sums else None
        n = L.gdr_layernorm_bwd_workspace_bytes(desc, 0, int(sums))
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        held.append((dx, db, ws, st))
        calls.append(lambda a=dx, b=db, w=ws, n=n, s=st: L.gdr_layernorm_bwd(
            desc, _p(x), _p(dy), None, _p(mean), _p(rstd), _p(a), None, _p(b), _p(w), n, s.cuda_stream))
    torch.cuda.synchronize()
    assert _at_once(L, calls, 3000) == set()
    torch.cuda.synchronize()
    for dx, db, _, _ in held:
        assert torch.equal(dx, ref["x"]) and (db is None or torch.equal(db, ref["bias"]))
