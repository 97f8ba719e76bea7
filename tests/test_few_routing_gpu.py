"""The few-token layer routes as moe_route_topk does, special logits included."""
import pytest
import torch

import activation_sparse_expert_amd as moe
from gpu_helpers import DEV
from test_few_gpu import make, new_trace
from test_linear_gpu import gen, normal

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def same(a, b):
    return torch.equal(a.view(torch.int32), b.view(torch.int32)) or \
        (torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)))


# what the bias of the experts named is: masked experts, all but one or all of them
# masked, fewer left than are chosen, the type's lowest value, one that takes all, NaN
SPECIAL = {"none": {}, "some masked": {0: -INF, 3: -INF}, "one left": {e: -INF for e in range(6) if e != 4},
           "all masked": {e: -INF for e in range(6)}, "lowest": {e: torch.finfo(torch.float32).min for e in range(5)},
           "one takes all": {2: INF}, "two take all": {2: INF, 5: INF}, "one NaN": {1: NAN},
           "all NaN": {e: NAN for e in range(6)}}


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("name", sorted(SPECIAL))
@pytest.mark.parametrize("T,E,k", [(1, 6, 3), (6, 6, 3), (20, 6, 6), (1, 70, 20), (9, 300, 5), (1, 300, 5)])
def test_choices_and_weights(T, E, k, name, renorm):
    g = gen(81 + T)
    L = make(g, 1024, 40, E, k, 1, torch.bfloat16, renorm, bias=True)
    for e, b in SPECIAL[name].items():
        L.router_bias[e] = b
        if E > 6:
            L.router_bias[e + E - 6] = b
    x = normal(g, (T, 1024), 1.0, torch.bfloat16)
    tr = new_trace(L, T)
    y = moe.layer_forward_few(L, x, trace=tr)
    r = moe.route_topk(x, L.router_w, k, renormalize=renorm, bias=L.router_bias)
    idx, w = r["topk_idx"], r["topk_w"]
    torch.cuda.synchronize()
    assert torch.equal(tr["topk_idx"], idx)
    assert same(tr["topk_w"], w)
    # a token whose weights are numbers has an output of numbers
    assert torch.equal(torch.isfinite(y).all(1), torch.isfinite(w).all(1))
