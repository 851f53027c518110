"""A process's first call of an operator may be one that a graph captures: what
the library allocates on a device at first does not end the capture."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

START = """
import torch
import int8_quantized_gb300 as q
dev, graph = torch.device("cuda:0"), torch.cuda.CUDAGraph()
torch.cuda.set_device(0)
g = torch.Generator(device=dev)
g.manual_seed(0)
rand = lambda *s: torch.randn(s, device=dev, generator=g)
pool = rand(4, 2, 16, 64).to(torch.bfloat16)
cache = q.KVCache(pool, rand(4, 2, 16, 64).to(torch.bfloat16))
table = torch.arange(4, dtype=torch.int32, device=dev).view(1, 4)
index, seq = torch.arange(3, dtype=torch.int32, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
x, u, w = rand(3, 2, 64), torch.rand(3, device=dev, generator=g), torch.ones(64, device=dev)
logits, one = rand(3, 500), torch.full((1,), 40, dtype=torch.int32, device=dev)
B, s, A = torch.randint(0, 256, (64, 4, 16), dtype=torch.uint8, device=dev, generator=g), rand(64, 4), rand(20, 128).bfloat16()
"""

CALLS = {
    "sample": ("out = torch.full((3,), -7, dtype=torch.int32, device=dev)", "q.sample(logits, u, out)"),
    "kv_append": ("out = torch.zeros_like(x)", "q.kv_append(cache, table, seq, index, x, x, q=x, q_out=out, k_norm=w, q_norm=w)"),
    "paged_attention": ("out = torch.zeros((1, 4, 64), device=dev); "
                        "work = torch.empty(q.paged_attention_workspace_size(cache, table, 4), dtype=torch.uint8, device=dev)",
                        "q.paged_attention(cache, table, one, x[:1].repeat(1, 2, 1), out, workspace=work)"),
    "matmul_nbits": ("out = torch.zeros((20, 64), dtype=torch.bfloat16, device=dev); m = q.MatMulNBits(B, s, 128, 32)",
                     "m.forward(A, out)"),
}

END = """
first = out.clone()
graph.replay()
q.sync_status()
got = out.clone()
out.copy_(first)
{call}
q.sync_status()
assert torch.equal(got, out) and not torch.equal(got, first)
print("same")
"""


@pytest.mark.parametrize("name", sorted(CALLS))
def test_the_first_call_is_captured(dev, name):
    before, call = CALLS[name]
    code = START + before + "\ntorch.cuda.synchronize()\nwith torch.cuda.graph(graph):\n    " + call + END.format(call=call)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=120)
    assert r.returncode == 0 and r.stdout.endswith("same\n"), r.stderr[-2000:]
