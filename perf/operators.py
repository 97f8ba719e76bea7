"""Cases, plain forms and 64-bit values of the linear layer and the few-token MoE layer.

``run`` is one pass: with ``own`` false from elementary torch operations in 32
bits (router logits in 64: a choice next to a border must not turn on a
rounding), with ``own`` true through the library's public calls.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _linear(name, T, k, n, dt, act="none", gated=False, bias=False, residual=False, out=None):
    return {"name": name, "op": "linear", "T": T, "k": k, "n": n, "dt": dt, "act": act, "gated": gated,
            "bias": bias, "residual": residual, "out": out or dt}


def _few(name, T, d, f, E, k, S, dt, renorm=True, bias=False, residual=True):
    return {"name": name, "op": "few", "T": T, "d": d, "f": f, "E": E, "k": k, "S": S, "dt": dt,
            "renorm": renorm, "bias": bias, "residual": residual}


def listed():
    return [
        # the projections of the tiny expert's size: nothing but latency
        _linear("linear tiny", 1, 256, 704, "f16", act="silu", bias=True),
        # one decoded token through the gated half of a dense SwiGLU FFN
        _linear("linear token gated", 1, 4096, 14336, "bf16", act="silu", gated=True),
        # a decode batch through its down projection, added to the residual stream
        _linear("linear batch down", 16, 14336, 4096, "f16", residual=True),
        # scores over a vocabulary for a few sequences, kept in 32 bits
        _linear("linear scores", 5, 4096, 32000, "bf16", out="f32"),
        # a ragged batch, an odd number of outputs, the classic GELU MLP
        _linear("linear ragged", 77, 2056, 1411, "f16", act="gelu", bias=True, residual=True),
        # a short prompt through a square projection with bias and residual
        _linear("linear prompt", 300, 4096, 4096, "bf16", bias=True, residual=True),
        # a long prompt through the gated half of a dense FFN: bound by the matrix cores
        _linear("linear prefill gated", 4096, 4096, 14336, "bf16", act="silu", gated=True),
        # the smallest layer: nothing but latency
        _few("few tiny", 1, 256, 704, 4, 2, 1, "f16"),
        # one decoded token through a fine-grained layer (64 routed top-6 and 2 shared experts)
        _few("few fine token", 1, 2048, 1408, 64, 6, 2, "f16", bias=True),
        # a decode batch through it: most experts are chosen by some token
        _few("few fine batch", 32, 2048, 1408, 64, 6, 2, "bf16", renorm=False, bias=True),
        # four sequences through a layer of eight wide experts, top-2
        _few("few wide experts", 4, 4096, 14336, 8, 2, 0, "f16"),
        # sizes that fill no tile: tokens, channels, experts
        _few("few ragged", 13, 1000, 712, 17, 3, 1, "bf16", bias=True, residual=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    dt = rng.choice(["f16", "bf16"])
    if rng.random() < 0.55:
        while True:
            T, k, n = _log(rng, 1, 4096), 8 * _log(rng, 8, 1792), _log(rng, 1, 32000)
            gated = rng.random() < 0.4
            cost = T * k * n * (2 if gated else 1)
            if 4096 <= k * n and cost <= 2 * 4096 * 4096 * 14336 and k * n <= 4096 * 32000:
                break
        act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"] if gated else
                         ["none", "none", "relu", "gelu", "gelu_tanh", "silu"])
        out = "f32" if rng.random() < 0.2 else dt
        return {"op": "linear", "T": T, "k": k, "n": n, "dt": dt, "act": act, "gated": gated,
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.5, "out": out}
    while True:
        T, d, f = _log(rng, 1, 32), 8 * _log(rng, 32, 512), 8 * _log(rng, 16, 1792)
        E, S = _log(rng, 2, 128), rng.choice([0, 0, 1, 2])
        k = rng.randint(1, min(8, E))
        if T * (k + S) * d * f <= 32 * 8 * 2048 * 1408 and (E + S) * d * f <= 8 * 4096 * 14336:
            break
    return {"op": "few", "T": T, "d": d, "f": f, "E": E, "k": k, "S": S, "dt": dt,
            "renorm": rng.random() < 0.5, "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DT[case["dt"]]

    def normal(shape, std, dtype=dt):
        return torch.randn(shape, generator=g, device=DEV, dtype=dtype).mul_(std)

    s = dict(case)
    T = case["T"]
    if case["op"] == "linear":
        # hidden states of unit scale, weights at the scale that keeps them so
        k, n = case["k"], case["n"]
        s["x"] = normal((T, k), 1.0)
        s["w"] = normal((n, k), k ** -0.5)
        s["w_gate"] = normal((n, k), k ** -0.5) if case["gated"] else None
        s["b"] = normal((n,), 0.5, torch.float32) if case["bias"] else None
        s["b_gate"] = normal((n,), 0.5, torch.float32) if case["bias"] and case["gated"] else None
        s["r"] = normal((T, n), 1.0, DT[case["out"]]) if case["residual"] else None
        return s
    d, f, E, S = case["d"], case["f"], case["E"], case["S"]
    s["x"] = normal((T, d), 1.0)
    s["router"] = normal((E, d), 2.0 * d ** -0.5)
    # popular and unpopular experts, as a trained router has them
    s["rb"] = normal((E,), 1.0, torch.float32) if case["bias"] else None
    s["gate"] = normal((E + S, f, d), d ** -0.5)
    s["up"] = normal((E + S, f, d), d ** -0.5)
    s["down"] = normal((E + S, d, f), f ** -0.5)
    s["r"] = normal((T, d), 1.0) if case["residual"] else None
    return s


def _act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * 0.7071067811865476))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(0.7978845608028654 * (v + 0.044715 * v * v * v)))
    return v


def _linear_plain(s):
    x = s["x"].float()
    a = x @ s["w"].float().t()
    if s["b"] is not None:
        a = a + s["b"]
    if s["gated"]:
        g = x @ s["w_gate"].float().t()
        if s["b_gate"] is not None:
            g = g + s["b_gate"]
        a = _act(g, s["act"]) * a
    else:
        a = _act(a, s["act"])
    if s["r"] is not None:
        a = a + s["r"].float()
    return a.to(DT[s["out"]])


def _choose(lg, k, renorm):
    """The k largest logits of each row, ties to the lower index, and their weights."""
    top, idx = torch.sort(lg, dim=1, descending=True, stable=True)
    e = torch.exp(lg - top[:, :1])
    chosen = torch.gather(e, 1, idx[:, :k])
    den = chosen if renorm else e
    return idx[:, :k], chosen / den.sum(1, keepdim=True)


def _few_plain(s):
    T, E, S, k = s["T"], s["E"], s["S"], s["k"]
    lg = s["x"].double() @ s["router"].double().t()
    if s["rb"] is not None:
        lg = lg + s["rb"].double()
    idx, w = _choose(lg, k, s["renorm"])
    w = w.float()
    every = torch.cat([idx, torch.arange(E, E + S, device=DEV).expand(T, S)], 1)
    scale = torch.cat([w, torch.ones((T, S), device=DEV)], 1)
    x = s["x"].float()[:, None, :, None]
    g = torch.matmul(s["gate"][every].float(), x)[..., 0]
    u = torch.matmul(s["up"][every].float(), x)[..., 0]
    h = _act(g, "silu") * u
    o = torch.matmul(s["down"][every].float(), h[..., None])[..., 0]
    y = (o * scale[..., None]).sum(1)
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(s["x"].dtype), "experts": idx.to(torch.int32), "weights": w}


def _linear_own(s):
    import activation_sparse_expert_amd as moe
    lin = moe.Linear(s["w"], bias=s["b"], w_gate=s["w_gate"], bias_gate=s["b_gate"], act=s["act"])
    return moe.linear_forward(lin, s["x"], residual=s["r"], out_dtype=DT[s["out"]])


def _few_own(s):
    import activation_sparse_expert_amd as moe
    layer = moe.Layer(d=s["d"], f=s["f"], E=s["E"], S=s["S"], k=s["k"], renormalize=s["renorm"],
                      router_w=s["router"], router_bias=s["rb"], up_q=None, up_sz=None, gate_t=s["gate"],
                      down=None, thresholds=None, up_dense=s["up"], down_dense=s["down"])
    tr = {"topk_idx": torch.empty((s["T"], s["k"]), dtype=torch.int32, device=DEV),
          "topk_w": torch.empty((s["T"], s["k"]), dtype=torch.float32, device=DEV)}
    y = moe.layer_forward_few(layer, s["x"], residual=s["r"], out_dtype=s["x"].dtype, trace=tr)
    return {"y": y, "experts": tr["topk_idx"], "weights": tr["topk_w"]}


def run(state):
    if own:
        return _linear_own(state) if state["op"] == "linear" else _few_own(state)
    return _linear_plain(state) if state["op"] == "linear" else _few_plain(state)


def work(case):
    T = case["T"]
    if case["op"] == "linear":
        k, n, m = case["k"], case["n"], 2 if case["gated"] else 1
        osz = 4 if case["out"] == "f32" else 2
        return {"bytes": 2 * T * k + 2 * m * n * k + (4 * m * n if case["bias"] else 0)
                + osz * T * n * (2 if case["residual"] else 1), "flops": 2 * m * T * n * k}
    d, f, E, S, k = case["d"], case["f"], case["E"], case["S"], case["k"]
    # experts that T tokens choose when each is as likely as the next
    chosen = E * (1 - (1 - k / E) ** T) + S
    return {"bytes": round(chosen * 6 * d * f + 2 * E * d + 2 * T * d * (3 if case["residual"] else 2) + 8 * T * k),
            "flops": 6 * T * (k + S) * d * f + 2 * T * E * d}


def _act64(v, act):
    if act == "none":
        return v
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2.0))
    return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))


def _linear_exact(s):
    out = torch.empty((s["T"], s["n"]), dtype=torch.float64, device=DEV)
    x = s["x"].double().t().contiguous()
    for j in range(0, s["n"], 4096):
        a = torch.mm(s["w"][j:j + 4096].double(), x)
        if s["b"] is not None:
            a += s["b"][j:j + 4096, None].double()
        if s["gated"]:
            g = torch.mm(s["w_gate"][j:j + 4096].double(), x)
            if s["b_gate"] is not None:
                g += s["b_gate"][j:j + 4096, None].double()
            a = a * _act64(g, s["act"])
        else:
            a = _act64(a, s["act"])
        out[:, j:j + 4096] = a.t()
    return out if s["r"] is None else out + s["r"].double()


def _few_exact(s):
    T, E, S, k = s["T"], s["E"], s["S"], s["k"]
    lg = (s["x"].double()[:, None, :] * s["router"].double()[None]).sum(-1)
    if s["rb"] is not None:
        lg += s["rb"].double()
    rows = lg.cpu().tolist()
    y = torch.zeros((T, s["d"]), dtype=torch.float64, device=DEV)
    takes, experts, weights = {}, [], []
    for t, row in enumerate(rows):
        best = sorted(range(E), key=lambda e: (-row[e], e))[:k]
        top = row[best[0]]
        den = sum(math.exp(row[e] - top) for e in (best if s["renorm"] else range(E)))
        experts.append(best)
        weights.append([math.exp(row[e] - top) / den for e in best])
        for e, w in zip(best, weights[-1]):
            takes.setdefault(e, []).append((t, w))
    for e in range(E, E + S):
        takes[e] = [(t, 1.0) for t in range(T)]
    for e, of in takes.items():
        at = torch.tensor([t for t, _ in of], device=DEV)
        xt = s["x"][at].double().t().contiguous()
        h = _act64(torch.mm(s["gate"][e].double(), xt), "silu") * torch.mm(s["up"][e].double(), xt)
        o = torch.mm(s["down"][e].double(), h).t()
        y.index_add_(0, at, o * torch.tensor([w for _, w in of], dtype=torch.float64, device=DEV)[:, None])
    if s["r"] is not None:
        y += s["r"].double()
    return {"y": y, "experts": torch.tensor(experts, dtype=torch.int32, device=DEV),
            "weights": torch.tensor(weights, dtype=torch.float64, device=DEV)}


def exact(case, seed):
    s = prepare(case, seed)
    return _linear_exact(s) if case["op"] == "linear" else _few_exact(s)
