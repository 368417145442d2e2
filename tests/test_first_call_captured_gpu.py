"""The first call of a process may be inside a stream capture: each cache operator in a process of
its own, captured before anything else has set the device up."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = '''
import sys
import torch
from tensor_core_gemm_fp16_b200 import binding


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


lens, add, ring, free, tables = i32([0, 3]), i32([4, 1]), i32([0, 8]), i32(list(range(8))), \\
    i32([[0] * 4] * 2)
kc, vc = torch.zeros(2, 8, 16, 2, 64, device="cuda").half()
k, v = torch.randn(2, 5, 2, 64, device="cuda").half()
q = torch.randn(5, 8, 64, device="cuda").half()
parents, starts, slots = i32([-1, 0, 0, 1, -1]), i32([0, 4, 5]), torch.arange(5, device="cuda")
call = {
    "plan": lambda: binding.cache_plan(lens, add, ring, free, tables, 16, 5).slots,
    "write": lambda: binding.cache_write(k, v, slots, kc, vc)[0],
    "mask": lambda: binding.tree_mask(parents, starts, 64)[0],
    "attention": lambda: binding.tree_attention(q, k, v, kc, vc, tables, lens, starts),
}[sys.argv[1]]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = call()
graph.replay()
torch.cuda.synchronize()
assert torch.equal(captured, call())
stream = torch.cuda.current_stream().cuda_stream
assert binding.tg_gemm_check_error(stream) == binding.TG_OK
a = torch.randn(128, 64, device="cuda").half()
assert binding.gemm(a, a.t().contiguous()).shape == (128, 128)
print("fine")
'''


@pytest.mark.parametrize("what", ["plan", "write", "mask", "attention"])
def test_first_call_of_a_process_in_a_capture(what):
    env = dict(os.environ, PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, "-c", PROGRAM, what], cwd=ROOT, env=env, timeout=120,
                       capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]
