"""A streamed linear layer whose workgroups are more than one launch can have."""
import pytest
import torch

import activation_sparse_expert_amd as moe
from dense_helpers import check
from gpu_helpers import DEV
from test_linear_gpu import gen, normal, want

pytestmark = pytest.mark.gpu


def test_more_workgroups_than_a_launch_has():
    """2080 tokens at a row stride past 2^21 (which streams at any T) by 2^23 gated outputs
    of 256 inputs: 1.7e7 workgroups of 256 threads, past 2^32 threads.  51 GB; every token at some outputs."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    g = gen(61)
    T, k, n, stride = 2080, 256, 1 << 23, (1 << 21) + 8
    f16 = torch.float16
    w, wg = (torch.randn((n, k), generator=g, device=DEV, dtype=f16).mul_(k ** -0.5) for _ in range(2))
    x = torch.empty(T * stride, dtype=f16, device=DEV).view(T, stride)[:, :k]
    x.copy_(normal(g, (T, k), 1.0, f16))
    y = torch.empty((T, n), dtype=f16, device=DEV)
    y[:, ::4096] = float("nan")
    moe.linear_forward(moe.Linear(w, w_gate=wg, act="silu"), x, y=y)
    cols = torch.cat([torch.arange(0, n, 4096, device=DEV), torch.tensor([1, n - 33, n - 1], device=DEV)])
    part = moe.Linear(w[cols].contiguous(), w_gate=wg[cols].contiguous(), act="silu")
    check(y[:, cols], *want(part, x, None, f16), "sampled outputs")
