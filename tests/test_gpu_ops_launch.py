"""Launches of the 4-bit products, read from a captured graph: they follow the
call's shape alone."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# launches(call): (grid, threads, dynamic LDS bytes) of each kernel that `call` puts on the current stream
LAUNCHES = """
import ctypes, torch
import mxfp4_weight_expert_amd as moe

class Dim3(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in "xyz"]

class Kernel(ctypes.Structure):  # hipKernelNodeParams
    _fields_ = [("block", Dim3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p), ("grid", Dim3),
                ("params", ctypes.c_void_p), ("lds", ctypes.c_uint32)]

def launches(call):
    hip = ctypes.CDLL([l.split()[-1] for l in open("/proc/self/maps") if "libamdhip64" in l][0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    graph, n = ctypes.c_void_p(g.raw_cuda_graph()), ctypes.c_size_t()
    assert hip.hipGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert hip.hipGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        k = Kernel()
        assert hip.hipGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(k)) == 0
        out.append((k.grid.x, k.block.x, k.lds))
    return out

def w4(M, N, K, E=1, **kw):
    s = moe.W4Shape(M=M, N=N, K=K, E=E, **kw)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(E, (N + 15) // 16 * 16, K // 2, dtype=torch.uint8, device="cuda")
    int4 = s.format == "int4"
    sc = torch.zeros(E, N, K // s.group, dtype=torch.bfloat16 if int4 else torch.uint8, device="cuda")
    out = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    if E == 1:
        return lambda: moe.w4_linear(x, w, sc, s, out=out)
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda").clamp(max=M)
    return lambda: moe.w4_grouped_linear(x, off, w, sc, s, out=out)
"""


def _child(code):
    r = subprocess.run([sys.executable, "-c", LAUNCHES + code], capture_output=True, text=True, timeout=100, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout.splitlines()[-1]


def test_launch_does_not_depend_on_products_that_ran_before():
    # two kernels with the same LDS bytes, of 512 and 256 threads: what the one lets a
    # CU hold says nothing about the other
    one, many = "w4(1, 7168, 2048)", "w4(1024, 768, 2304, E=896)"
    for first, second in ((one, many), (many, one)):
        print(f"[ops] launch of {second} after {first}", flush=True)
        alone = _child(f"print(launches({second}))")
        after = _child(f"{first}()\nprint(launches({second}))")
        assert after == alone


def test_tiles_of_64_rows_leave_room_for_two_blocks():
    # 64 KB of tokens a block: with a wave reading all of K, the scales of 128 weight
    # rows (24 KB here) keep a second block off the CU, where a fourth of them does not
    call = 'w4(64, 129279, 4096, format="int4", group=64)'
    print(f"[ops] launch of {call}", flush=True)
    (_, threads, lds), = eval(_child(f"print(launches({call}))"))
    assert threads == 256 and 2 * (lds + 8224) <= 160 << 10  # 8224: the table of experts' tiles
