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


def test_after_a_device_reset():
    """A process that resets its own context and goes on: the status query, and the scan's tensor maps."""
    import subprocess
    import sys
    code = """
import ctypes, glob, os, sys
import torch                                     # for its libcudart alone: no context of torch's is made
from recurrent_state_memory_b200 import gdr as G
L = G.lib()
rt = ctypes.CDLL([l.split()[-1] for l in open("/proc/self/maps") if "libcudart" in l][0])
def buffers(n):
    p = [ctypes.c_void_p() for _ in range(n)]
    for q in p:
        assert rt.cudaMalloc(ctypes.byref(q), ctypes.c_size_t(1 << 16)) == 0
        assert rt.cudaMemset(q, 0, ctypes.c_size_t(1 << 16)) == 0
    return p
d = G.scan_desc(2, 100, 8, torch.bfloat16, torch.bfloat16, torch.bfloat16)
for _ in range(3):
    x, g, h, S, parent = buffers(5)
    assert L.gdr_scan_fwd(ctypes.byref(d), x, g, None, None, h, None, None, None) == 0, L.gdr_last_error_detail()
    assert L.gdr_query_device_status(None) == 0, L.gdr_last_error_detail()
    assert rt.cudaMemset(parent, 9, ctypes.c_size_t(16)) == 0
    r = G.ReorderDesc(1, 1, 4, 64)
    assert L.gdr_state_reorder(ctypes.byref(r), S, parent, None) == 0
    assert L.gdr_query_device_status(None) == G.GDR_ERR_INDEX
    assert L.gdr_query_device_status(None) == 0
    assert rt.cudaDeviceReset() == 0
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
