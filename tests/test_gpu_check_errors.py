"""gm_check_device_errors beside the attention calls, whose kernels have an error word of their own: in a
process of its own, since the word is read from the first of these calls on."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys, time
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import sparse_dynamic_routing_b200 as gm

def check_us():
    took = []
    for _ in range(300):
        t = time.perf_counter()
        gm.gm_check_device_errors()
        took.append((time.perf_counter() - t) * 1e6)
    return sorted(took)[150]

def raises():
    try:
        gm.gm_check_device_errors()
    except gm.GMIndexRangeError:
        return True
    return False

torch.zeros(1, device="cuda")
before = check_us()
k = torch.ones(1, 1, 1, 64, device="cuda").bfloat16()
pool = [torch.zeros(2, 1, 16, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
scales = [torch.ones(2, 1, device="cuda") for _ in range(2)]
table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
lens = torch.zeros(1, dtype=torch.int32, device="cuda")
s = torch.cuda.Stream()
s.wait_stream(torch.cuda.current_stream())
with torch.cuda.stream(s):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):  # the first attention call only ever runs as a replay
        gm.gm_kv8_append(k, k, *pool, *scales, table, lens)
torch.cuda.current_stream().wait_stream(s)
assert not raises()
table.fill_(7)  # a page outside the pool: not written, reported
graph.replay()
assert raises() and not raises()
graph.replay()
assert raises()
table.fill_(1)
graph.replay()
assert not raises()
after = check_us()
print("US", before, after)
"""


def test_the_attention_calls_errors_are_found_and_the_others_pay_nothing():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    run = subprocess.run([sys.executable, "-c", PROGRAM.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-1000:]
    before, after = map(float, run.stdout.split("US")[1].split())
    # one copy from the device against two (measured: 19 and 31 us)
    assert before < 0.9 * after, (before, after)
