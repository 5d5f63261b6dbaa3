"""fp4_mx_check reads the error words of the kernels that a process has launched, so a program of
products alone pays for one; and a linear layer's give-up is seen however it was launched."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from test_gpu_fp4_product import operand
from test_gpu_ops import G, dev  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


COST = """
import sys, time
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import loss_scaling_master_gb300 as G
q, s = G.fp4_mx_buffers(256, 256)
G.fp4_quant_mx(torch.randn(256, 256, device="cuda"), q, s)
out = torch.empty(256, 256, device="cuda")
G.fp4_product_mx(q, s, q, s, 256, out)
torch.cuda.synchronize()
took = {{G.fp4_mx_check: [], G.amp_noalloc_check: []}}
for _ in range(400):
    for f, t in took.items():
        t0 = time.perf_counter()
        f()
        t.append(time.perf_counter() - t0)
print(*[sorted(t)[200] for t in took.values()])
"""


def test_a_check_of_products_costs_one_read(G, dev):
    """It takes about as long as amp_noalloc_check, which reads one word of the device too; three words
    take 2.4 times as long."""
    r = subprocess.run([sys.executable, "-c", COST.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    mine, one = map(float, r.stdout.split())
    assert mine < 1.7 * one, (mine, one)


FIRST = """
import sys
sys.path.insert(0, {root!r})
import torch
import loss_scaling_master_gb300 as G
# 1.0 = code 2 with scale 127: A, B of ones, k = 32 (the scales' padding counts for nothing)
m, n, k = {m}, {n}, 32
ones = lambda r: (torch.full((r, 16), 0x22, dtype=torch.uint8, device="cuda"),
                  torch.full((512 * -(-r // 128),), 127, dtype=torch.uint8, device="cuda"))
a, b = ones(m), ones(n)
out = torch.zeros(m, n, device="cuda")
s = torch.cuda.Stream()
s.wait_stream(torch.cuda.current_stream())
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=s):
    G.fp4_linear_mx(*a, *b, k, out, residual=out)
g.replay()
g.replay()
torch.cuda.synchronize()
assert (out == 64.0).all(), out
G.fp4_mx_check()
print("right")
"""


@pytest.mark.parametrize("m,n", [(5, 200), (2049, 5120)])
def test_the_first_call_of_a_process_is_captured(m, n):
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, m=m, n=n)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "right", r.stderr[-2000:]


@pytest.mark.parametrize("m,n", [(5, 200), (2049, 5122)])
def test_a_replayed_give_up_is_seen(G, dev, m, n):
    """The launch was captured; each replay sets the word, each check clears it."""
    k = 600
    a, b = operand(G, m, k, 1)[:2], operand(G, n, k, 2, 0.02)[:2]
    out = torch.empty(m, n, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        st = G.ops._load().fp4_linear_mx_selftest(
            *[x.data_ptr() for x in (*a, *b)], m, n, k, None, 1, -1, None, out.data_ptr(), 1, None, None, 2, 1, 22,
            ctypes.c_void_p(s.cuda_stream))
    assert st == 0
    G.fp4_mx_check()
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        with pytest.raises(G.AmpError) as e:
            G.fp4_mx_check()
        assert e.value.status == -6 and out.isnan().any()
        G.fp4_mx_check()
