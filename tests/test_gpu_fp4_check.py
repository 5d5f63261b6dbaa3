"""fp4_mx_check reads one error word for the products and the linear layers, whichever kernel gave up,
and the linear layer's way to that word is open from its first call, captured or not."""
import os
import subprocess
import sys
import time

import pytest
import torch

from test_gpu_fp4_product import operand
from test_gpu_ops import G, dev  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_check_costs_one_read(G, dev):
    """After products and linear layers on one CTA a tile and on pairs, a check takes about as long as
    amp_noalloc_check, which reads one word of the device too; three reads take 2.4 times as long."""
    for m, n, k in ((3, 200, 300), (2049, 5121, 96)):
        a, sa, _ = operand(G, m, k, 1)
        b, sb, _ = operand(G, n, k, 2, 0.02)
        out = torch.empty(m, n, device=dev)
        G.fp4_product_mx(a, sa, b, sb, k, out)
        G.fp4_linear_mx(a, sa, b, sb, k, out, kind="gelu")
    torch.cuda.synchronize()
    took = {G.fp4_mx_check: [], G.amp_noalloc_check: []}
    for _ in range(400):
        for f, t in took.items():
            t0 = time.perf_counter()
            f()
            t.append(time.perf_counter() - t0)
    mid = [sorted(t)[200] for t in took.values()]
    assert mid[0] < 1.7 * mid[1], mid


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
