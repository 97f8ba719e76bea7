"""Calls of one kernel from several host threads whose launches ask for different
amounts of LDS above 64 KB: one thread's limit must not undercut another's."""
import threading

import pytest
import torch

import activation_sparse_expert_amd as moe
from gpu_helpers import DEV
from test_few_gpu import make
from test_linear_gpu import gen, layer, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def together(calls, rounds):
    """Each call in a thread and on a stream of its own, `rounds` times; the last results."""
    out, errors = [None] * len(calls), []
    start = threading.Barrier(len(calls))

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                start.wait()
                for _ in range(rounds):
                    out[i] = calls[i]()
            stream.synchronize()
        except Exception as e:                           # reported by the test's own thread
            errors.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    return out


def test_streamed_linear_layers():
    """32 tokens: 8 slices of k in a workgroup (144 KB) where outputs are few, else 4 (72 KB)."""
    g = gen(51)
    x = normal(g, (32, 2048), 1.0, torch.bfloat16)
    calls = [lambda lin=layer(g, n, 2048, torch.bfloat16): moe.linear_forward(lin, x) for n in (704, 9000, 512, 12000)]
    alone = [c() for c in calls]
    torch.cuda.synchronize()
    got = together(calls, 400)
    assert all(torch.equal(a, b) for a, b in zip(alone, got))


def test_few_token_layers():
    """1024 experts, ranked in 66 to 150 KB; the down product's rows likewise."""
    g = gen(52)
    L = make(g, 64, 40, 1024, 4, 0, torch.bfloat16)
    xs = [normal(g, (T, 64), 1.0, torch.bfloat16) for T in (14, 20, 26, 32)]
    calls = [lambda x=x: moe.layer_forward_few(L, x) for x in xs]
    alone = [c() for c in calls]
    torch.cuda.synchronize()
    got = together(calls, 400)
    assert all(torch.equal(a, b) for a, b in zip(alone, got))
