"""Cases, plain forms and 64-bit values of three operators around the layers of a decode step: the
linear layer on 8-bit integers, rows to 8 bits and back, and the norms between two blocks.

``run`` is one pass: with ``own`` false from elementary torch operations in 32 bits (the quotients
that 8-bit codes are rounded from in 64: a code next to a border must not turn on a rounding),
with ``own`` true through the library's public calls.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.int8}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "i8": 1}


def _linear(name, T, k, n, x, out, act="none", gated=False, bias=False, residual=False):
    """x: the type of the tokens; i8: codes with a scale for each token, else the call makes them."""
    return {"name": name, "op": "linear", "T": T, "k": k, "n": n, "x": x, "out": out, "act": act, "gated": gated,
            "bias": bias, "residual": residual}


def _rows(name, T, k, x, out):
    return {"name": name, "op": "rows", "T": T, "k": k, "x": x, "out": out}


def _norm(name, T, d, kind, h, block=None, out="f16", w="f16", bias=False, post=False, gate="none", offset=False,
          scales=(1.0, 1.0)):
    """h: the type of the residual stream; block: that of the block's output (None: only a norm);
    gate: none, a factor for each channel, or one for each token and channel."""
    return {"name": name, "op": "norm", "T": T, "d": d, "kind": kind, "h": h, "block": block or "none", "out": out, "w": w,
            "bias": bias, "post": post, "gate": gate, "offset": offset, "rs": scales[0], "bs": scales[1]}


def listed():
    return [
        # the projections of the tiny expert's size: nothing but latency
        _linear("linear tiny", 1, 256, 704, "i8", "f16", act="silu", bias=True),
        # one decoded token, in 16 bits, through the gated half of a dense SwiGLU FFN
        _linear("linear token gated", 1, 4096, 14336, "bf16", "bf16", act="silu", gated=True),
        # a decode batch through its down projection, added to the residual stream
        _linear("linear batch down", 16, 14336, 4096, "i8", "f16", residual=True),
        # a ragged batch in 16 bits, an odd number of outputs, the classic GELU MLP
        _linear("linear ragged", 77, 2064, 1411, "f16", "f16", act="gelu", bias=True, residual=True),
        # a short prompt through a square projection with bias and residual
        _linear("linear prompt", 300, 4096, 4096, "i8", "bf16", bias=True, residual=True),
        # a long prompt through the gated half of a dense FFN: bound by the matrix cores
        _linear("linear prefill gated", 4096, 4096, 14336, "i8", "bf16", act="silu", gated=True),
        # one token's hidden channels to 8 bits and back: nothing but latency
        _rows("rows token", 1, 14336, "bf16", "bf16"),
        # a long prompt's hidden channels to 8 bits and back
        _rows("rows prompt", 4096, 14336, "bf16", "bf16"),
        # between two blocks of a decoded token: the block added to the stream, the next one's RMS norm
        _norm("norm token", 1, 4096, "rms", "f16", "f16"),
        # a norm of each head of a long prompt: many short rows
        _norm("norm heads", 131072, 128, "rms", "bf16", out="bf16", w="bf16"),
        # sizes that fill no vector: layer norms before and after, a stream in 32 bits, a gate for each token
        _norm("norm ragged", 77, 1411, "layer", "f32", "bf16", out="bf16", w="f32", bias=True, post=True, gate="token"),
        # a long prompt between two blocks with norms on both sides, a gate for each channel, the next product on 8 bits
        _norm("norm prompt to 8 bits", 4096, 6144, "rms", "bf16", "bf16", out="i8", w="bf16", post=True, gate="channel",
              offset=True, scales=(1.0, 0.5)),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    dt = rng.choice(["f16", "bf16"])
    kind = rng.choice(["linear", "linear", "rows", "norm", "norm"])
    if kind == "linear":
        while True:
            T, k, n = _log(rng, 1, 4096), 16 * _log(rng, 4, 896), _log(rng, 1, 32000)
            gated = rng.random() < 0.4
            if 4096 <= k * n <= 4096 * 32000 and T * k * n * (2 if gated else 1) <= 2 * 4096 * 4096 * 14336:
                break
        act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"] if gated else
                         ["none", "none", "relu", "gelu", "gelu_tanh", "silu"])
        return {"op": "linear", "T": T, "k": k, "n": n, "x": rng.choice(["i8", "i8", dt, dt, "f32"]),
                "out": "f32" if rng.random() < 0.2 else dt, "act": act, "gated": gated,
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}
    if kind == "rows":
        while True:
            T, k = _log(rng, 1, 8192), _log(rng, 8, 16384)
            if T * k <= 4096 * 14336:
                break
        x = rng.choice([dt, dt, "f32"])
        return {"op": "rows", "T": T, "k": k, "x": x, "out": rng.choice([x, dt])}
    while True:
        T, d = _log(rng, 1, 131072), _log(rng, 8, 16384)
        if T * d <= 4096 * 6144:
            break
    h, block = rng.choice([dt, dt, "f32"]), rng.choice(["none", dt, dt, dt, "f32"])
    bare = block == "none"
    return {"op": "norm", "T": T, "d": d, "kind": rng.choice(["rms", "layer"]), "h": h, "block": block,
            "out": rng.choice([dt, dt, "f32", "i8"]), "w": rng.choice([dt, "f32"]), "bias": rng.random() < 0.4,
            "post": not bare and rng.random() < 0.5, "gate": "none" if bare else rng.choice(["none", "channel", "token"]),
            "offset": rng.random() < 0.3, "rs": rng.choice([1.0, 1.0, 0.75]), "bs": rng.choice([1.0, 1.0, 0.25])}


def _codes(x):
    """Codes and scales of rows: q = 127 x / max |x| rounded to nearest, ties to even; scale = max |x| / 127."""
    top = x.abs().amax(1, keepdim=True).double()
    q = torch.round(x.double() * 127 / torch.where(top > 0, top, torch.ones_like(top)))
    return q.to(torch.int8), (top / 127).float()[:, 0]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(shape, std, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=DEV, dtype=dtype).mul_(std)

    s = dict(case)
    T = case["T"]
    if case["op"] == "linear":
        # hidden states of unit scale, weights at the scale that keeps them so, with a scale for each channel
        k, n = case["k"], case["n"]
        s["sx"] = None
        if case["x"] == "i8":
            s["tokens"], s["sx"] = _codes(normal((T, k), 1.0))
        else:
            s["tokens"] = normal((T, k), 1.0, DT[case["x"]])
        s["w"], s["sw"] = _codes(normal((n, k), k ** -0.5, torch.float16))
        s["wg"], s["sg"] = _codes(normal((n, k), k ** -0.5, torch.float16)) if case["gated"] else (None, None)
        s["b"] = normal((n,), 0.5) if case["bias"] else None
        s["bg"] = normal((n,), 0.5) if case["bias"] and case["gated"] else None
        s["r"] = normal((T, n), 1.0, DT[case["out"]]) if case["residual"] else None
        return s
    if case["op"] == "rows":
        # SiLU(g) u of unit g and u, as a gated layer's hidden channels are spread
        u = normal((T, case["k"]), 1.0, DT[case["x"]])
        v = normal((T, case["k"]), 1.0, DT[case["x"]])
        s["tokens"] = u.mul_(v.mul_(torch.sigmoid(v)))
        return s
    d, wt = case["d"], DT[case["w"]]
    s["r"] = normal((T, d), 2.0, DT[case["h"]])
    s["o"] = normal((T, d), 0.5, DT[case["block"]]) if case["block"] != "none" else None
    shape = {"none": None, "channel": (d,), "token": (T, d)}[case["gate"]]
    s["g"] = normal(shape, 0.5, DT[case["block"]]) if shape else None
    at = 0.0 if case["offset"] else 1.0
    s["pre_w"] = normal((d,), 0.2, wt).add_(at)
    s["pre_b"] = normal((d,), 0.2, wt) if case["bias"] else None
    s["post_w"] = normal((d,), 0.2, wt).add_(at) if case["post"] else None
    s["post_b"] = normal((d,), 0.2, wt) if case["bias"] and case["post"] else None
    return s


EPS = 1e-6


def _act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.erfc(v * -0.7071067811865476)
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(0.7978845608028654 * (v + 0.044715 * v * v * v)))
    return v


def _linear_plain(s):
    q, sx = (s["tokens"], s["sx"]) if s["x"] == "i8" else _codes(s["tokens"])
    q = q.float()
    a = (q @ s["w"].float().t()) * (sx[:, None] * s["sw"])
    if s["b"] is not None:
        a = a + s["b"]
    if s["gated"]:
        g = (q @ s["wg"].float().t()) * (sx[:, None] * s["sg"])
        if s["bg"] is not None:
            g = g + s["bg"]
        a = _act(g, s["act"]) * a
    else:
        a = _act(a, s["act"])
    if s["r"] is not None:
        a = a + s["r"].float()
    return a.to(DT[s["out"]])


def _rows_plain(s):
    q, scale = _codes(s["tokens"])
    return {"values": (q.float() * scale[:, None]).to(DT[s["out"]]), "scale": scale}


def _plain_norm(v, kind, w, b, offset):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    v = v * (w.float() + 1 if offset else w.float())
    return v if b is None else v + b.float()


def _norm_plain(s):
    v = s["r"].float()
    if s["o"] is not None:
        o = s["o"].float()
        if s["post"]:
            o = _plain_norm(o, s["kind"], s["post_w"], s["post_b"], s["offset"])
        if s["g"] is not None:
            o = o * s["g"].float()
        v = s["rs"] * v + s["bs"] * o
    elif s["rs"] != 1.0:
        v = s["rs"] * v
    n = _plain_norm(v, s["kind"], s["pre_w"], s["pre_b"], s["offset"])
    out = {} if s["o"] is None else {"stream": v.to(DT[s["h"]])}
    if s["out"] != "i8":
        return {**out, "normed": n.to(DT[s["out"]])}
    q, scale = _codes(n)
    return {**out, "normed": (q.float() * scale[:, None]).to(torch.bfloat16), "scale": scale}


def _linear_own(s):
    import activation_sparse_expert_amd as moe
    lin = moe.LinearQ8(s["w"], s["sw"], bias=s["b"], w_gate=s["wg"], gate_scale=s["sg"], bias_gate=s["bg"], act=s["act"])
    return moe.linear_q8_forward(lin, s["tokens"], x_scale=s["sx"], residual=s["r"], out_dtype=DT[s["out"]])


def _rows_own(s):
    import activation_sparse_expert_amd as moe
    q, scale = moe.quantize_rows(s["tokens"])
    return {"values": moe.dequantize_rows(q, scale, out_dtype=DT[s["out"]]), "scale": scale}


def _norm_own(s):
    import activation_sparse_expert_amd as moe
    norm = moe.Norm(s["d"], kind=s["kind"], eps=EPS, w=s["pre_w"], b=s["pre_b"], post=s["post"], post_w=s["post_w"],
                    post_b=s["post_b"], offset=s["offset"], residual_scale=s["rs"], block_scale=s["bs"])
    y, n, scale = moe.norm_forward(norm, s["r"], s["o"], gate=s["g"], out_dtype=DT[s["out"]])
    out = {} if s["o"] is None else {"stream": y}
    if s["out"] != "i8":
        return {**out, "normed": n}
    return {**out, "normed": moe.dequantize_rows(n, scale, out_dtype=torch.bfloat16), "scale": scale}


def run(state):
    op = state["op"]
    if own:
        return _linear_own(state) if op == "linear" else _rows_own(state) if op == "rows" else _norm_own(state)
    return _linear_plain(state) if op == "linear" else _rows_plain(state) if op == "rows" else _norm_plain(state)


def work(case):
    T = case["T"]
    if case["op"] == "linear":
        k, n, m = case["k"], case["n"], 2 if case["gated"] else 1
        scales = 4 * m * n + (4 * T if case["x"] == "i8" else 0)
        return {"bytes": SIZE[case["x"]] * T * k + m * n * k + scales + (4 * m * n if case["bias"] else 0)
                + SIZE[case["out"]] * T * n * (2 if case["residual"] else 1), "flops": 2 * m * T * n * k}
    if case["op"] == "rows":
        return {"bytes": T * case["k"] * (SIZE[case["x"]] + SIZE[case["out"]]) + 4 * T, "flops": 6 * T * case["k"]}
    d, bare = case["d"], case["block"] == "none"
    values = SIZE[case["h"]] * (1 if bare else 2) + (2 if case["out"] == "i8" else SIZE[case["out"]])
    gates = {"none": 0, "channel": d, "token": T * d}[case["gate"]]
    weights = (2 if case["post"] else 1) * (2 if case["bias"] else 1) * d * SIZE[case["w"]]
    block = 0 if bare else SIZE[case["block"]] * (T * d + gates)
    return {"bytes": T * d * values + block + weights + (4 * T if case["out"] == "i8" else 0),
            "flops": T * d * (16 if case["post"] else 8)}


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


def _stand_for(x):
    """(whole numbers, step) in 64 bits of rows held in 8 bits."""
    v = x.double()
    most = v.abs().max(dim=1, keepdim=True).values
    return (127 * v / most.clamp(min=1e-300)).round(), most / 127


def _linear_exact(s):
    q, step = (s["tokens"].double(), s["sx"].double()[:, None]) if s["x"] == "i8" else _stand_for(s["tokens"])
    out = torch.empty((s["T"], s["n"]), dtype=torch.float64, device=DEV)
    at = (q * step).t().contiguous()
    for j in range(0, s["n"], 4096):
        a = torch.mm(s["w"][j:j + 4096].double(), at) * s["sw"][j:j + 4096, None].double()
        if s["b"] is not None:
            a += s["b"][j:j + 4096, None].double()
        if s["gated"]:
            g = torch.mm(s["wg"][j:j + 4096].double(), at) * s["sg"][j:j + 4096, None].double()
            if s["bg"] is not None:
                g += s["bg"][j:j + 4096, None].double()
            a = a * _act64(g, s["act"])
        else:
            a = _act64(a, s["act"])
        out[:, j:j + 4096] = a.t()
    return out if s["r"] is None else out + s["r"].double()


def _norm64(v, kind, w, b, offset):
    c = v - v.sum(1, keepdim=True) / v.shape[1] if kind == "layer" else v
    out = c / torch.sqrt((c ** 2).sum(1, keepdim=True) / v.shape[1] + EPS) * ((1.0 if offset else 0.0) + w.double())
    return out if b is None else out + b.double()


def _norm_exact(s):
    v = s["rs"] * s["r"].double()
    out = {}
    if s["o"] is not None:
        c = s["o"].double()
        if s["post"]:
            c = _norm64(c, s["kind"], s["post_w"], s["post_b"], s["offset"])
        v = v + s["bs"] * (c if s["g"] is None else s["g"].double() * c)
        out["stream"] = v
    out["normed"] = _norm64(v, s["kind"], s["pre_w"], s["pre_b"], s["offset"])
    if s["out"] == "i8":
        whole, step = _stand_for(out["normed"])
        out["normed"], out["scale"] = whole * step, step[:, 0]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _linear_exact(s)
    if case["op"] == "norm":
        return _norm_exact(s)
    whole, step = _stand_for(s["tokens"])
    return {"values": whole * step, "scale": step[:, 0]}
