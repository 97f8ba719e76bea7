"""A process whose first norm is captured into a graph (run by test_norm_rows_gpu.py)."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import torch  # noqa: E402

import activation_sparse_expert_amd as moe  # noqa: E402

x = torch.randn(700, 520, device="cuda", dtype=torch.bfloat16)
out = torch.zeros_like(x)
moe.lib()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    moe.norm_forward(moe.Norm(520), x, out=out)
graph.replay()
torch.cuda.synchronize()
again = moe.norm_forward(moe.Norm(520), x)[1]
assert torch.equal(out, again) and bool(out.any())
print("first norm in a capture: ok")
