"""The status word of the 8-bit products called without a workspace.  It is made
once per device, so each case runs in a process of its own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import torch
import moe_routing_expert_fp32_b200 as moe
moe.lib()
def operands(E):
    w = torch.ones(E, 128, 128, device="cuda").to(torch.float8_e4m3fn)
    return (torch.ones(8, 128, device="cuda").to(torch.float8_e4m3fn),
            torch.ones(8, 1, device="cuda"), w, torch.ones(E, 1, 1, device="cuda"))
xq, xs, w, ws = operands(2)
off = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
y = torch.empty(8, 128, dtype=torch.bfloat16, device="cuda")
z = torch.empty_like(y)
def linear(out): return moe.linear_fp8(xq, xs, w[0], ws[0], out=out)
def grouped(out): return moe.grouped_linear_fp8(xq, xs, off, w, ws, out=out)
wk = moe.workspace(256)  # the kernels are loaded; the shared word is not made by this
moe.linear_fp8(xq, xs, w[0], ws[0], out=y, ws=wk)
moe.grouped_linear_fp8(xq, xs, off, w, ws, out=y, ws=wk)
torch.cuda.synchronize()
"""


def run(body, call):
    r = subprocess.run([sys.executable, "-c", SETUP + f"call = {call}\n" + body], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]


@pytest.mark.parametrize("call", ["linear", "grouped"])
def test_no_memory_of_another_stream_is_cleared(call):
    """Stream A frees a small tensor whose reader is still queued and makes the
    first call; stream B, which does not wait for A, makes the second while A
    still sleeps.  What A reads is as it was."""
    run("""
a, b = torch.cuda.Stream(), torch.cuda.Stream()
with torch.cuda.stream(a):
    small = [torch.full((64,), 7, dtype=torch.int32, device="cuda") for _ in range(8)]
    torch.cuda._sleep(1_500_000_000)
    read = [t.clone() for t in small]
    del small
    call(y)
with torch.cuda.stream(b):
    call(z)
b.synchronize()
assert not a.query(), "the sleep was too short to show anything"
a.synchronize()
for t in read:
    assert (t == 7).all(), t
assert (y == 128).all() and (z == 128).all()
""", call)


@pytest.mark.parametrize("call", ["linear", "grouped"])
def test_nothing_of_the_allocator_is_kept(call):
    run("""
before = torch.cuda.memory_allocated()
call(y)
torch.cuda.synchronize()
assert torch.cuda.memory_allocated() == before
""", call)


@pytest.mark.parametrize("call", ["linear", "grouped"])
def test_first_call_inside_a_capture(call):
    """The first call of a process may be captured: nothing of the graph's pool is
    kept, and calls after the graph is gone are as always."""
    run("""
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    call(y)
g.replay()
torch.cuda.synchronize()
assert (y == 128).all()
g.reset()
del g
torch.cuda.empty_cache()
call(z)
torch.cuda.synchronize()
assert (z == 128).all()
""", call)
