"""The MoE layer of plain 16-bit experts for a few tokens
(moe_layer_forward_few) against 64 bits, alone and in a stack with the linear
layer."""
import pytest
import torch

import activation_sparse_expert_amd as moe
from dense_helpers import U, check, choose64, few64, linear64
from gpu_helpers import DEV, Guarded, say
from test_linear_gpu import gen, normal

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def make(g, d, f, E, k, S, dt, renorm=True, bias=False, rdt=None):
    return moe.Layer(d=d, f=f, E=E, S=S, k=k, renormalize=renorm,
                     router_w=normal(g, (E, d), 2 * d ** -0.5, rdt or dt),
                     router_bias=normal(g, (E,), 1.0, torch.float32) if bias else None,
                     up_q=None, up_sz=None, thresholds=None, down=None,
                     gate_t=normal(g, (E + S, f, d), d ** -0.5, dt),
                     up_dense=normal(g, (E + S, f, d), d ** -0.5, dt),
                     down_dense=normal(g, (E + S, d, f), f ** -0.5, dt))


def new_trace(L, T):
    i, fl = torch.int32, torch.float32
    return dict(topk_idx=torch.empty((T, L.k), dtype=i, device=DEV), topk_w=torch.empty((T, L.k), dtype=fl, device=DEV),
                logits=torch.empty((T, L.E), dtype=fl, device=DEV), expert_count=torch.empty(L.E, dtype=i, device=DEV),
                eam_row=torch.full((L.E,), 5, dtype=i, device=DEV),
                expert_dense=torch.full((L.E,), 7, dtype=torch.uint8, device=DEV))


def check_routing(L, x, tr):
    """Choices as 64 bits choose (up to logits that fp32 cannot tell apart),
    weights, and the counts that follow."""
    lg, idx, w = choose64(x, L.router_w, L.router_bias, L.k, L.renormalize)
    tol = (L.d / 8 + 64) * U * (x.double().abs() @ L.router_w.double().abs().t().contiguous() +
                                (0 if L.router_bias is None else L.router_bias.double().abs()))
    assert bool(((tr["logits"].double() - lg).abs() <= tol).all())
    got = tr["topk_idx"].long()
    for t in range(x.shape[0]):
        chosen = got[t].tolist()
        assert len(set(chosen)) == L.k and min(chosen) >= 0 and max(chosen) < L.E
    near = 2 * float(tol.max())
    assert bool((torch.gather(lg, 1, idx) - torch.gather(lg, 1, got)).abs().max() <= near)
    e = torch.exp(lg - lg.max(1, keepdim=True).values)
    c = torch.gather(e, 1, got)
    w64 = c / (c if L.renormalize else e).sum(1, keepdim=True)
    assert bool(((tr["topk_w"].double() - w64).abs() <= w64 * (2 * near + 32 * U)).all())
    count = torch.bincount(got.flatten(), minlength=L.E)
    assert torch.equal(tr["expert_count"].long(), count)
    assert torch.equal(tr["eam_row"].long(), count + 5)
    assert torch.equal(tr["expert_dense"].bool(), count > 0)


def run(L, x, residual=None, out=torch.float32):
    T = x.shape[0]
    y = Guarded((T, L.d), out)
    ws = Guarded((moe.workspace_size(moe.OP_LAYER_FEW, T, L.d, L.f, L.E, L.k, L.S),), torch.uint8)
    tr = new_trace(L, T)
    moe.layer_forward_few(L, x, residual=residual, y=y.t, trace=tr, ws=ws.t)
    torch.cuda.synchronize()
    y.check("y")
    ws.check("workspace")
    return y.t, tr


SHAPES = [  # T, d, f, E, k, S
    (1, 8, 8, 1, 1, 0), (1, 256, 704, 4, 2, 1), (1, 2048, 1408, 64, 6, 2), (2, 264, 72, 5, 5, 0),
    (4, 1000, 712, 17, 3, 1), (13, 520, 328, 40, 4, 2), (16, 4096, 256, 8, 2, 0), (17, 136, 1000, 9, 2, 1),
    (31, 2048, 264, 64, 6, 2), (32, 512, 96, 130, 8, 0), (32, 64, 40, 1024, 1, 1), (32, 128, 64, 3, 1, 3),
    (1, 72, 200, 1000, 3, 0), (1, 64, 40, 40, 20, 1), (3, 64, 40, 70, 17, 0), (20, 96, 136, 2, 2, 1),
    (20, 2048, 264, 4, 2, 1), (10, 2056, 264, 4, 2, 1), (5, 4096, 72, 3, 1, 2),
    # the limits: T (k + S), experts, inputs, choices worked out by every workgroup
    (32, 64, 40, 1024, 63, 1), (32, 128, 64, 600, 32, 32), (32, 16384, 72, 6, 2, 0), (1, 64, 24, 1024, 16, 0),
    (1, 64, 40, 5, 2, 700), (8, 8, 16, 512, 64, 0)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,d,f,E,k,S", SHAPES)
def test_against_64_bits(T, d, f, E, k, S, dt):
    for renorm, bias, res, out in ((True, False, False, "f32"), (False, True, True, dt)):
        say(f"few T={T} d={d} f={f} E={E} k={k} S={S} {dt} renorm={renorm} bias={bias} residual={res} -> {out}")
        g = gen(T + d + f + E + renorm)
        L = make(g, d, f, E, k, S, DT[dt], renorm, bias)
        x = normal(g, (T, d), 1.0, DT[dt])
        r = normal(g, (T, d), 1.0, DT[out]) if res else None
        y, tr = run(L, x, r, DT[out])
        check_routing(L, x, tr)
        check(y, *few64(x, L.gate_t, L.up_dense, L.down_dense, tr["topk_idx"], tr["topk_w"], S, r, DT[out]), "y")
        again = moe.layer_forward_few(L, x, residual=r, out_dtype=DT[out])
        torch.cuda.synchronize()
        assert torch.equal(y, again), "two runs differ"


@pytest.mark.parametrize("T", [1, 6, 20])
@pytest.mark.parametrize("rdt", [torch.float32, torch.float16, torch.bfloat16])
def test_router_types(T, rdt):
    g = gen(3 + T)
    L = make(g, 320, 64, 12, 3, 0, torch.bfloat16, rdt=rdt, bias=True)
    x = normal(g, (T, 320), 1.0, torch.bfloat16)
    y, tr = run(L, x)
    check_routing(L, x, tr)
    check(y, *few64(x, L.gate_t, L.up_dense, L.down_dense, tr["topk_idx"], tr["topk_w"], 0), "y")


@pytest.mark.parametrize("T", [1, 9, 32])
@pytest.mark.parametrize("E,k", [(6, 2), (64, 6), (200, 3)])
def test_equal_logits_go_to_the_lower_expert(T, E, k):
    g = gen(5)
    L = make(g, 512, 64, E, k, 0, torch.float16)
    L.router_w[:] = L.router_w[:1]                   # every expert the same
    x = normal(g, (T, 512), 1.0, torch.float16)
    _, tr = run(L, x)
    assert tr["topk_idx"].tolist() == [list(range(k))] * T


@pytest.mark.parametrize("T", [3, 24])
def test_one_expert_takes_all(T):
    """A bias sends every token to expert 4: all other experts stay empty."""
    g = gen(6)
    L = make(g, 264, 136, 9, 1, 0, torch.bfloat16, bias=True)
    L.router_bias[4] = 1e4
    x = normal(g, (T, 264), 1.0, torch.bfloat16)
    y, tr = run(L, x)
    assert bool((tr["topk_idx"] == 4).all()) and int(tr["expert_count"][4]) == T
    check(y, *few64(x, L.gate_t, L.up_dense, L.down_dense, tr["topk_idx"], tr["topk_w"], 0), "y")


@pytest.mark.parametrize("T", [8, 30])
def test_infinities_reach_only_their_tokens(T):
    """Infinite weights of one expert and a NaN in one token's x leave the other
    tokens' outputs as they were."""
    g = gen(8)
    L = make(g, 200, 104, 6, 2, 0, torch.float16)
    x = normal(g, (T, 200), 1.0, torch.float16)
    clean, tr = run(L, x)
    hit = (tr["topk_idx"] == 3).any(1)
    assert bool(hit.any()) and not bool(hit.all())
    L.gate_t[3, 5] = float("inf")
    L.up_dense[3, 7] = float("nan")
    L.down_dense[3, :, 1] = float("inf")
    y, tr2 = run(L, x)
    assert torch.equal(tr["topk_idx"], tr2["topk_idx"])
    assert torch.equal(y[~hit], clean[~hit])
    assert not bool(torch.isfinite(y[hit]).any())
    t0 = int(torch.nonzero(~hit)[0])
    x[t0, 199] = float("nan")
    # all-NaN logits choose experts 0 and 1, which may add an expert to the call's
    # list and so move the borders between partial sums: not the same bits, but
    # the same 64-bit values within the same bound
    y2, tr3 = run(L, x)
    rest = [t for t in range(T) if t != t0 and not bool(hit[t])]
    assert tr3["topk_idx"][t0].tolist() == [0, 1] and torch.equal(tr3["topk_idx"][rest], tr["topk_idx"][rest])
    want, bound = few64(x[rest], L.gate_t, L.up_dense, L.down_dense, tr["topk_idx"][rest], tr["topk_w"][rest], 0)
    check(y2[rest], want, bound, "other tokens")
    assert bool(torch.isnan(y2[t0]).all())


def test_large_h_keeps_its_infinity():
    """fp16 layers: a SiLU(g) u past 65504 makes its token's outputs infinite,
    not NaN, and nothing else."""
    g = gen(9)
    L = make(g, 64, 32, 2, 1, 0, torch.float16)
    L.gate_t[:] = 0
    L.up_dense[:] = 0
    L.gate_t[:, 3, 0] = 1
    L.up_dense[:, 3, 0] = 1
    L.down_dense[:] = 1
    x = torch.zeros((3, 64), dtype=torch.float16, device=DEV)
    x[0, 0], x[1, 0], x[2, 0] = 2.0, 400.0, 200.0
    y, tr = run(L, x)
    assert bool((y[1] == float("inf")).all())
    keep = [0, 2]
    want, bound = few64(x[keep], L.gate_t, L.up_dense, L.down_dense, tr["topk_idx"][keep], tr["topk_w"][keep], 0)
    check(y[keep], want, bound, "finite tokens")


def test_in_place_residual():
    g = gen(10)
    L = make(g, 256, 128, 8, 2, 1, torch.bfloat16)
    x = normal(g, (5, 256), 1.0, torch.bfloat16)
    want, bound = None, None
    stream = x.clone()
    y, tr = run(L, x)
    want, bound = few64(x, L.gate_t, L.up_dense, L.down_dense, tr["topk_idx"], tr["topk_w"], 1, x, torch.bfloat16)
    moe.layer_forward_few(L, stream, residual=stream, y=stream)
    check(stream, want, bound, "x as residual and output")


@pytest.mark.parametrize("T", [1, 12, 32])
def test_graph_replays_follow_their_inputs(T):
    g = gen(12)
    L = make(g, 512, 264, 16, 4, 1, torch.float16, bias=True)
    x = normal(g, (T, 512), 1.0, torch.float16)
    y = torch.empty((T, 512), dtype=torch.float16, device=DEV)
    ws = moe.new_workspace(moe.workspace_size(moe.OP_LAYER_FEW, T, 512, 264, 16, 4, 1))
    moe.layer_forward_few(L, x, residual=x, y=y, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.layer_forward_few(L, x, residual=x, y=y, ws=ws)
    for i in range(4):
        x.copy_(normal(g, (T, 512), 1.0, torch.float16))
        eager = moe.layer_forward_few(L, x, residual=x, out_dtype=torch.float16)
        y.zero_()
        ws.fill_(0xFF)                               # a workspace holds nothing between calls
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager), f"replay {i}"


def test_two_graphs_share_a_workspace():
    """Graphs of both operators that follow each other on one stream may use one workspace."""
    g = gen(23)
    bf = torch.bfloat16
    d = 1024
    L = make(g, d, 328, 12, 3, 1, bf)
    lin = moe.Linear(normal(g, (d, 4 * d), d ** -0.5 / 2, bf))
    x, z = normal(g, (9, d), 1.0, bf), normal(g, (200, 4 * d), 1.0, bf)
    split = moe.workspace_size(moe.OP_LINEAR, 200, 4 * d, d)
    assert split > 0
    ws = moe.new_workspace(max(moe.workspace_size(moe.OP_LAYER_FEW, 9, d, 328, 12, 3, 1), split))
    y, v = torch.empty((9, d), dtype=bf, device=DEV), torch.empty((200, d), dtype=bf, device=DEV)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    with torch.cuda.graph(graphs[0]):
        moe.layer_forward_few(L, x, y=y, ws=ws)
    with torch.cuda.graph(graphs[1]):
        moe.linear_forward(lin, z, y=v, ws=ws)
    for i in range(3):
        x.copy_(normal(g, (9, d), 1.0, bf))
        z.copy_(normal(g, (200, 4 * d), 1.0, bf))
        a, b = moe.layer_forward_few(L, x, out_dtype=bf), moe.linear_forward(lin, z, out_dtype=bf)
        for graph in graphs + graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, a) and torch.equal(v, b), f"replay {i}"


def test_two_streams_with_their_own_workspaces():
    g = gen(13)
    L = make(g, 1024, 512, 16, 2, 1, torch.bfloat16)
    xs = [normal(g, (T, 1024), 1.0, torch.bfloat16) for T in (3, 25)]
    alone = [moe.layer_forward_few(L, x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    out = [None, None]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            for _ in range(5):
                out[i] = moe.layer_forward_few(L, xs[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, out))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_agrees_with_the_dense_path(dt):
    """moe_layer_forward's dense path on the same experts: its h has 16 bits, so
    its y may be off by eps / 2 of |h| through |W^down| more than this one's."""
    g = gen(14)
    d, f, E, k, S, T = 512, 256, 8, 2, 1, 24
    L = make(g, d, f, E, k, S, DT[dt])
    x = normal(g, (T, d), 1.0, DT[dt])
    y, tr = run(L, x)
    L.down = L.down_dense.transpose(1, 2).contiguous()
    L.up_q = torch.zeros((E + S, f, d // 4), dtype=torch.uint8, device=DEV)
    L.up_sz = torch.zeros((E + S, f, d // 64, 2), dtype=torch.int16, device=DEV)
    L.thresholds = torch.zeros(E + S, device=DEV)
    tr2 = {"topk_idx": torch.empty_like(tr["topk_idx"])}
    yd = moe.layer_forward(L, x, path=moe.PATH_DENSE, trace=tr2)
    assert torch.equal(tr["topk_idx"], tr2["topk_idx"])
    want, bound = few64(x, L.gate_t, L.up_dense, L.down_dense, tr["topk_idx"], tr["topk_w"], S)
    eps = torch.finfo(DT[dt]).eps / 2
    size = torch.zeros((T, d), dtype=torch.float64, device=DEV)
    for t in range(T):
        for e, w in [(int(tr["topk_idx"][t, s]), float(tr["topk_w"][t, s])) for s in range(k)] + \
                [(E + i, 1.0) for i in range(S)]:
            gg, u = L.gate_t[e].double() @ x[t].double(), L.up_dense[e].double() @ x[t].double()
            size[t] += w * (L.down_dense[e].double().abs() @ (gg * torch.sigmoid(gg) * u).abs())
    check(yd, y.double(), 2 * bound + 1.01 * eps * size, "dense path")


@pytest.mark.parametrize("T", [1, 7, 32])
def test_a_stack_of_dense_and_moe_layers(T):
    """Two FFN halves as a model runs them: a dense SwiGLU FFN with its residual
    added by the down product, then an MoE layer with its residual; each step
    against 64 bits from what the step before it wrote."""
    g = gen(15 + T)
    d, fd, f = 512, 1376, 264
    dt = torch.bfloat16
    up = moe.Linear(normal(g, (fd, d), d ** -0.5, dt), w_gate=normal(g, (fd, d), d ** -0.5, dt), act="silu")
    down = moe.Linear(normal(g, (d, fd), fd ** -0.5, dt))
    L = make(g, d, f, 16, 4, 1, dt, bias=True)
    x = normal(g, (T, d), 1.0, dt)
    h = moe.linear_forward(up, x, out_dtype=dt)
    x1 = moe.linear_forward(down, h, residual=x, out_dtype=dt)
    tr = new_trace(L, T)
    y = moe.layer_forward_few(L, x1, residual=x1, out_dtype=dt, trace=tr)
    torch.cuda.synchronize()
    check(h, *linear64(x, up.w, wg=up.w_gate, act="silu", out=dt), "gate/up")
    check(x1, *linear64(h, down.w, residual=x, out=dt), "down")
    check_routing(L, x1, tr)
    check(y, *few64(x1, L.gate_t, L.up_dense, L.down_dense, tr["topk_idx"], tr["topk_w"], 1, x1, dt), "moe")
