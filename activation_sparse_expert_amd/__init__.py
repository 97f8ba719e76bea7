"""Python binding of libmoeffn (activation-sparse MoE expert FFN, MI355X / gfx950).

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libmoeffn.so``.  PyTorch provides device memory and the current
stream.  If the shared library has not been built, every call raises.
"""
from __future__ import annotations

import ctypes as C
import functools
import os
from dataclasses import dataclass
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
# MOEFFN_LIB names another build of the same sources (the sanitizer build)
LIB_PATH = os.environ.get("MOEFFN_LIB") or os.path.join(HERE, "libmoeffn.so")

MOE_F16, MOE_BF16, MOE_F32, MOE_I8 = 0, 1, 2, 3
PATH_SPARSE, PATH_DENSE, PATH_AUTO, PATH_MIXED = 0, 1, 2, 3
OP_EXPERT, OP_ROUTE, OP_LAYER, OP_CALIBRATE, OP_EAMC, OP_EXPERT_BITS = 0, 1, 2, 3, 4, 5
OP_LINEAR, OP_LAYER_FEW, OP_LINEAR_Q8 = 6, 7, 8
ACT = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
NORM = {"rms": 0, "layer": 1}

STATUS = {0: "MOE_OK", -1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_UNSUPPORTED",
          -3: "MOE_ERR_ALIGNMENT", -4: "MOE_ERR_WORKSPACE", -5: "MOE_ERR_HIP"}

EXPORTED = ["moe_route_topk", "moe_expert_forward_sparse", "moe_layer_forward",
            "moe_workspace_size", "moe_workspace_init", "moe_pack_up_int2",
            "moe_materialize_up_bf16", "moe_status_string", "moe_calibrate_threshold",
            "moe_eamc_match", "moe_expert_forward_sparse_bits", "moe_pack_up_bits",
            "moe_build_sources_sha256", "moe_expert_forward_sparse_noalloc",
            "moe_noalloc_scratch_bytes", "moe_materialize_up", "moe_transpose_down",
            "moe_auto_dense_min", "moe_mixed_dense_min", "moe_layer_forward_few",
            "moe_linear_forward", "moe_linear_plan", "moe_linear_q8_forward", "moe_quantize_rows",
            "moe_dequantize_rows", "moe_norm_forward", "moe_linear_q8_plan"]


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


class ExpertView(C.Structure):
    _fields_ = [("up_q", C.c_void_p), ("up_sz", C.c_void_p), ("gate_t", C.c_void_p),
                ("down", C.c_void_p), ("threshold", C.c_float)]


class LayerDesc(C.Structure):
    _fields_ = [("d", C.c_int), ("f", C.c_int), ("n_routed", C.c_int), ("n_shared", C.c_int),
                ("top_k", C.c_int), ("renormalize", C.c_int), ("wdt", C.c_int),
                ("router_w", C.c_void_p), ("rdt", C.c_int), ("router_bias", C.c_void_p),
                ("up_q", C.c_void_p), ("up_sz", C.c_void_p), ("gate_t", C.c_void_p),
                ("down", C.c_void_p), ("thresholds", C.c_void_p), ("up_dense", C.c_void_p),
                ("down_dense", C.c_void_p), ("density", C.c_float)]


class LayerTrace(C.Structure):
    _fields_ = [("topk_idx", C.c_void_p), ("topk_w", C.c_void_p), ("logits", C.c_void_p),
                ("expert_count", C.c_void_p), ("masks", C.c_void_p), ("eam_row", C.c_void_p),
                ("mask_bits", C.c_void_p), ("nnz", C.c_void_p), ("expert_dense", C.c_void_p)]


class LinearDesc(C.Structure):
    _fields_ = [("n", C.c_int), ("k", C.c_int), ("wdt", C.c_int), ("w", C.c_void_p),
                ("bias", C.c_void_p), ("w_gate", C.c_void_p), ("bias_gate", C.c_void_p),
                ("act", C.c_int)]


class LinearQ8Desc(C.Structure):
    _fields_ = [("n", C.c_int), ("k", C.c_int), ("w", C.c_void_p), ("w_scale", C.c_void_p), ("bias", C.c_void_p),
                ("w_gate", C.c_void_p), ("gate_scale", C.c_void_p), ("bias_gate", C.c_void_p), ("act", C.c_int)]


class NormDesc(C.Structure):
    _fields_ = [("d", C.c_int), ("kind", C.c_int), ("eps", C.c_float), ("wdt", C.c_int), ("w", C.c_void_p),
                ("b", C.c_void_p), ("post", C.c_int), ("post_w", C.c_void_p), ("post_b", C.c_void_p),
                ("offset", C.c_int), ("residual_scale", C.c_float), ("block_scale", C.c_float)]


_lib = None


def lib():
    """The loaded libmoeffn.  Raises if it has not been built, or if it was
    built from other sources than the ones in csrc/ (a stale binary)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libmoeffn.so not built ({LIB_PATH}); run __graft_entry__.build()")
        from .build import sources_sha256
        L = C.CDLL(LIB_PATH)
        L.moe_build_sources_sha256.restype = C.c_char_p
        L.moe_build_sources_sha256.argtypes = []
        built = L.moe_build_sources_sha256().decode()
        want = sources_sha256()
        if built != want:
            raise RuntimeError(f"libmoeffn.so is stale: built from sources {built[:16]}..., "
                               f"csrc/ now hashes to {want[:16]}...; run __graft_entry__.build()")
        P, I, Z = C.c_void_p, C.c_int, C.c_size_t
        L.moe_route_topk.restype = I
        L.moe_route_topk.argtypes = [P, I, I, I, P, I, P, I, I, I, P, P, P, P, P, P, P, Z, P]
        L.moe_expert_forward_sparse.restype = I
        L.moe_expert_forward_sparse.argtypes = [C.POINTER(ExpertView), I, I, I, P, I, I, P, I,
                                                P, I, P, P, P, P, P, Z, P]
        L.moe_layer_forward.restype = I
        L.moe_layer_forward.argtypes = [C.POINTER(LayerDesc), P, I, I, P, I, I,
                                        C.POINTER(LayerTrace), P, Z, P]
        L.moe_workspace_size.restype = Z
        L.moe_workspace_size.argtypes = [I, I, I, I, I, I, I]
        L.moe_workspace_init.restype = I
        L.moe_workspace_init.argtypes = [P, Z, P]
        L.moe_pack_up_int2.restype = I
        L.moe_pack_up_int2.argtypes = [P, I, I, I, P, P, P]
        L.moe_materialize_up_bf16.restype = I
        L.moe_materialize_up_bf16.argtypes = [P, P, I, I, P, P]
        L.moe_materialize_up.restype = I
        L.moe_materialize_up.argtypes = [P, P, I, I, I, P, P]
        L.moe_transpose_down.restype = I
        L.moe_transpose_down.argtypes = [P, I, I, I, P, P]
        L.moe_auto_dense_min.restype = I
        L.moe_auto_dense_min.argtypes = [C.POINTER(LayerDesc), I]
        L.moe_mixed_dense_min.restype = I
        L.moe_mixed_dense_min.argtypes = [C.POINTER(LayerDesc), I]
        L.moe_status_string.restype = C.c_char_p
        L.moe_status_string.argtypes = [I]
        L.moe_calibrate_threshold.restype = I
        L.moe_calibrate_threshold.argtypes = [P, C.c_longlong, C.c_double, P, P, Z, P]
        L.moe_expert_forward_sparse_noalloc.restype = I
        L.moe_expert_forward_sparse_noalloc.argtypes = [C.POINTER(ExpertView), I, I, I, P, I, I,
                                                        P, I, P, I, P, P, P, P, P]
        L.moe_noalloc_scratch_bytes.restype = Z
        L.moe_noalloc_scratch_bytes.argtypes = []
        L.moe_expert_forward_sparse_bits.restype = I
        L.moe_expert_forward_sparse_bits.argtypes = [C.POINTER(ExpertView), I, I, I, I, P, I, I,
                                                     P, I, P, I, P, P, P, P, P, Z, P]
        L.moe_pack_up_bits.restype = I
        L.moe_pack_up_bits.argtypes = [P, I, I, I, I, P, P, P]
        L.moe_eamc_match.restype = I
        L.moe_eamc_match.argtypes = [P, I, I, P, P, P, P, Z, P]
        L.moe_layer_forward_few.restype = I
        L.moe_layer_forward_few.argtypes = [C.POINTER(LayerDesc), P, I, I, P, P, I,
                                            C.POINTER(LayerTrace), P, Z, P]
        L.moe_linear_forward.restype = I
        L.moe_linear_forward.argtypes = [C.POINTER(LinearDesc), P, I, C.c_longlong, I, P,
                                         C.c_longlong, P, I, C.c_longlong, P, Z, P]
        N = C.c_longlong
        L.moe_linear_q8_forward.restype = I
        L.moe_linear_q8_forward.argtypes = [C.POINTER(LinearQ8Desc), P, I, N, P, I, P, N, P, I, N, P, Z, P]
        L.moe_linear_q8_plan.restype = I
        L.moe_linear_q8_plan.argtypes = [I, I, I, I, C.POINTER(I), C.POINTER(I)]
        L.moe_quantize_rows.restype = I
        L.moe_quantize_rows.argtypes = [P, I, N, I, I, P, N, P, P]
        L.moe_dequantize_rows.restype = I
        L.moe_dequantize_rows.argtypes = [P, N, P, I, I, P, I, N, P]
        L.moe_norm_forward.restype = I
        L.moe_norm_forward.argtypes = [C.POINTER(NormDesc), I, P, I, N, P, I, N, P, N, P, N, P, I, N, P, P]
        L.moe_linear_plan.restype = I
        L.moe_linear_plan.argtypes = [I, I, I, I, C.POINTER(I), C.POINTER(I)]
        _lib = L
    return _lib


def _check(st: int, what: str):
    if st != 0:
        raise MoeError(st, what)


def _dt(t) -> int:
    import torch
    m = {torch.float16: MOE_F16, torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}
    if t.dtype not in m:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return m[t.dtype]


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoeffn must be contiguous")
    return t.data_ptr()


def _stream():
    import torch
    return torch.cuda.current_stream().cuda_stream


def workspace_size(op: int, T: int, d: int, f: int = 0, E: int = 1, k: int = 1, S: int = 0) -> int:
    return int(lib().moe_workspace_size(op, T, d, f, E, k, S))


def new_workspace(nbytes: int, device="cuda"):
    """A zero-filled workspace tensor (uint8) of at least ``nbytes``."""
    import torch
    return torch.zeros(max(256, (nbytes + 255) // 256 * 256), dtype=torch.uint8, device=device)


def workspace_init(ws) -> None:
    _check(lib().moe_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream()),
           "moe_workspace_init")


@dataclass
class Expert:
    """One compressed expert on the device (layouts as in include/moeffn.h)."""
    up_q: "torch.Tensor"        # [f][d/4] uint8
    up_sz: "torch.Tensor"       # [f][d/64][2] int16/uint16 (fp16 bits)
    gate_t: "torch.Tensor"      # [f][d] fp16/bf16
    down: "torch.Tensor"        # [f][d] fp16/bf16
    threshold: float

    @property
    def d(self):
        return self.gate_t.shape[1]

    @property
    def f(self):
        return self.gate_t.shape[0]

    def view(self) -> ExpertView:
        return ExpertView(_ptr(self.up_q), _ptr(self.up_sz), _ptr(self.gate_t), _ptr(self.down),
                          float(self.threshold))


def expert_forward_sparse(expert: Expert, x, *, y=None, out_dtype=None, token_scale=None,
                          accumulate: bool = False, mask_out=None, v_out=None, mask_bits=None,
                          nnz=None, ws=None):
    """Algorithm 1 of the FloE review on x [T][d]; returns y [T][d].

    Optional exports: mask_out [T][f] uint8, v_out [T][f] fp32, mask_bits
    [T][f/64] int64 (bit l of word i = channel 64 i + l), nnz [T] int32."""
    import torch
    T, d = x.shape
    if y is None:
        y = torch.empty((T, d), dtype=out_dtype or torch.float32, device=x.device)
    if ws is None:
        ws = new_workspace(workspace_size(OP_EXPERT, T, d, expert.f), x.device)
    v = expert.view()
    st = lib().moe_expert_forward_sparse(
        C.byref(v), d, expert.f, _dt(expert.gate_t), _ptr(x), _dt(x), T, _ptr(token_scale),
        int(bool(accumulate)), _ptr(y), _dt(y), _ptr(mask_bits), _ptr(nnz), _ptr(mask_out),
        _ptr(v_out), _ptr(ws), ws.numel(), _stream())
    _check(st, "moe_expert_forward_sparse")
    return y


def expert_forward_sparse_noalloc(expert: Expert, x, *, y, token_scale=None,
                                  accumulate: bool = False, mask_out=None, v_out=None,
                                  mask_bits=None, nnz=None):
    """expert_forward_sparse through the allocation-free entry point: the
    library's static device scratch serves as the workspace, and the caller
    passes every output (y included), so nothing is allocated."""
    T, d = x.shape
    v = expert.view()
    st = lib().moe_expert_forward_sparse_noalloc(
        C.byref(v), d, expert.f, _dt(expert.gate_t), _ptr(x), _dt(x), T, _ptr(token_scale),
        int(bool(accumulate)), _ptr(y), _dt(y), _ptr(mask_bits), _ptr(nnz), _ptr(mask_out),
        _ptr(v_out), _stream())
    _check(st, "moe_expert_forward_sparse_noalloc")
    return y


def expert_forward_sparse_bits(expert: Expert, bits: int, x, *, y=None, out_dtype=None,
                               token_scale=None, accumulate: bool = False, mask_out=None,
                               v_out=None, mask_bits=None, nnz=None, ws=None):
    """Algorithm 1 with the up codes at ``bits`` (8, 4, 2 or 1) bits; y [T][d]."""
    import torch
    T, d = x.shape
    if y is None:
        y = torch.empty((T, d), dtype=out_dtype or torch.float32, device=x.device)
    if ws is None:
        ws = new_workspace(workspace_size(OP_EXPERT_BITS, T, d, expert.f), x.device)
    v = expert.view()
    st = lib().moe_expert_forward_sparse_bits(
        C.byref(v), int(bits), d, expert.f, _dt(expert.gate_t), _ptr(x), _dt(x), T,
        _ptr(token_scale), int(bool(accumulate)), _ptr(y), _dt(y), _ptr(mask_bits), _ptr(nnz),
        _ptr(mask_out), _ptr(v_out), _ptr(ws), ws.numel(), _stream())
    _check(st, "moe_expert_forward_sparse_bits")
    return y


def route_topk(x, router_w, k: int, *, renormalize: bool = True, bias=None, logits=False, ws=None):
    """Top-k routing and grouping; returns a dict of device tensors."""
    import torch
    T, d = x.shape
    E = router_w.shape[0]
    dev = x.device
    out = dict(topk_idx=torch.empty((T, k), dtype=torch.int32, device=dev),
               topk_w=torch.empty((T, k), dtype=torch.float32, device=dev),
               expert_count=torch.empty(E, dtype=torch.int32, device=dev),
               expert_offset=torch.empty(E + 1, dtype=torch.int32, device=dev),
               pair_by_expert=torch.empty(T * k, dtype=torch.int32, device=dev))
    if logits:
        out["logits"] = torch.empty((T, E), dtype=torch.float32, device=dev)
    if ws is None:
        ws = new_workspace(workspace_size(OP_ROUTE, T, d, 0, E, k), dev)
    st = lib().moe_route_topk(_ptr(x), _dt(x), T, d, _ptr(router_w), _dt(router_w), _ptr(bias), E,
                              k, int(bool(renormalize)), _ptr(out["topk_idx"]), _ptr(out["topk_w"]),
                              _ptr(out["expert_count"]), _ptr(out["expert_offset"]),
                              _ptr(out["pair_by_expert"]), _ptr(out.get("logits")), _ptr(ws),
                              ws.numel(), _stream())
    _check(st, "moe_route_topk")
    return out


@dataclass
class Layer:
    """One MoE layer: E routed + S shared experts at a fixed stride."""
    d: int
    f: int
    E: int
    S: int
    k: int
    renormalize: bool
    router_w: "torch.Tensor"      # [E][d]
    up_q: "torch.Tensor"          # [E+S][f][d/4]
    up_sz: "torch.Tensor"         # [E+S][f][d/64][2]
    gate_t: "torch.Tensor"        # [E+S][f][d]
    down: "torch.Tensor"          # [E+S][f][d]
    thresholds: "torch.Tensor"    # [E+S] fp32
    router_bias: Optional["torch.Tensor"] = None
    up_dense: Optional["torch.Tensor"] = None   # [E+S][f][d] in the weight type
    down_dense: Optional["torch.Tensor"] = None  # [E+S][d][f] W^down transposed
    density: float = 0.0                         # expected active fraction (AUTO, MIXED)

    def desc(self) -> LayerDesc:
        return LayerDesc(self.d, self.f, self.E, self.S, self.k, int(bool(self.renormalize)),
                         _dt(self.gate_t), _ptr(self.router_w), _dt(self.router_w),
                         _ptr(self.router_bias), _ptr(self.up_q), _ptr(self.up_sz),
                         _ptr(self.gate_t), _ptr(self.down), _ptr(self.thresholds),
                         _ptr(self.up_dense), _ptr(self.down_dense), float(self.density))

    def workspace_bytes(self, T: int) -> int:
        return workspace_size(OP_LAYER, T, self.d, self.f, self.E, self.k, self.S)

    def auto_dense_min(self, T: int) -> int:
        """MOE_PATH_AUTO's choice at T tokens: 1 when the call takes the dense
        path (every expert with tokens), 0 when it stays sparse."""
        desc = self.desc()
        return int(lib().moe_auto_dense_min(C.byref(desc), T))

    def mixed_dense_min(self, T: int) -> int:
        """Token count from which MOE_PATH_MIXED sends an expert to the dense
        path at T tokens (0: the call stays sparse)."""
        desc = self.desc()
        return int(lib().moe_mixed_dense_min(C.byref(desc), T))


def layer_forward(layer: Layer, x, *, path: int = PATH_SPARSE, y=None, out_dtype=None,
                  trace: Optional[dict] = None, ws=None):
    """Route and combine one layer on x [T][d]; returns y [T][d].

    ``trace`` may map any of topk_idx, topk_w, logits, expert_count, masks,
    mask_bits, nnz, expert_dense to preallocated device tensors that receive
    those exports,
    and eam_row to an int32 [E] device tensor that the call's per-expert counts
    are added into."""
    import torch
    T, d = x.shape
    if y is None:
        y = torch.empty((T, d), dtype=out_dtype or torch.float32, device=x.device)
    if ws is None:
        ws = new_workspace(layer.workspace_bytes(T), x.device)
    tr = None
    if trace:
        tr = LayerTrace(_ptr(trace.get("topk_idx")), _ptr(trace.get("topk_w")),
                        _ptr(trace.get("logits")), _ptr(trace.get("expert_count")),
                        _ptr(trace.get("masks")), _ptr(trace.get("eam_row")),
                        _ptr(trace.get("mask_bits")), _ptr(trace.get("nnz")),
                        _ptr(trace.get("expert_dense")))
    desc = layer.desc()
    st = lib().moe_layer_forward(C.byref(desc), _ptr(x), _dt(x), T, _ptr(y), _dt(y), path,
                                 C.byref(tr) if tr is not None else None, _ptr(ws), ws.numel(),
                                 _stream())
    _check(st, "moe_layer_forward")
    return y


@functools.lru_cache(maxsize=1024)
def _size_of(op: int, T: int, d: int, f: int, E: int, k: int, S: int) -> int:
    return workspace_size(op, T, d, f, E, k, S)


def _want(name, t, device, shape, dtype=None):
    """Checks that t, unless None, lies on the call's GPU with this shape (and type)."""
    if t is None:
        return
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, x on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _rows(name, t, align=1):
    """(data pointer, row stride) of a matrix whose rows are contiguous.  The
    stride of a single row means nothing and is taken as the row's length."""
    T, n = t.shape
    rs, cs = t.stride()
    if cs != 1 and n > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.data_ptr(), rs if T > 1 else -(-n // align) * align


def _workspace(torch, device, nbytes, ws):
    """(pointer, bytes) of a call's workspace: the caller's, or one from
    torch's allocator (not initialised), or none where the call needs none."""
    if ws is not None:
        if ws.device != device:
            raise ValueError(f"ws is on {ws.device}, x on {device}")
        return ws, _ptr(ws), ws.numel() * ws.element_size()
    if not nbytes:
        return None, None, 0
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr(), nbytes


def _call(torch, device, what, fn, *args):
    """fn(*args, stream) on the device's current stream, with the device current."""
    i = device.index
    if i == torch._C._cuda_getDevice():                 # (a tensor of the device exists: it is initialised)
        st = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(i):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    if st != 0:
        raise MoeError(st, what)


_TRACE_DTYPES = {"topk_idx": "int32", "topk_w": "float32", "logits": "float32", "expert_count": "int32",
                 "eam_row": "int32", "expert_dense": "uint8"}


def layer_forward_few(layer: Layer, x, *, residual=None, y=None, out_dtype=None,
                      trace: Optional[dict] = None, ws=None):
    """One layer of plain 16-bit experts on the few tokens (1 to 32) of a decode
    step, x [T][d]; returns y [T][d] = residual + the layer's output.

    Reads the layer's router, gate_t, up_dense and down_dense; its up_q, up_sz,
    down and thresholds may be None.  ``residual`` [T][d] has y's type and may be
    y.  ``trace`` maps any of topk_idx [T][k], topk_w [T][k], logits [T][E],
    expert_count [E], expert_dense [E] and eam_row [E] to device tensors as in
    layer_forward."""
    import torch
    if x.dim() != 2:
        raise ValueError("x must be [T][d]")
    device = x.device
    if device.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    T, d = x.shape
    E, S, f, k = layer.E, layer.S, layer.f, layer.k
    gate, up, down = layer.gate_t, layer.up_dense, layer.down_dense
    if layer.router_w is None or gate is None or up is None or down is None:
        raise ValueError("the layer needs router_w, gate_t, up_dense and down_dense")
    if d != layer.d:
        raise ValueError(f"x has {d} columns, the layer d = {layer.d}")
    wdt = gate.dtype
    _want("router_w", layer.router_w, device, (E, d))
    _want("router_bias", layer.router_bias, device, (E,), torch.float32)
    _want("gate_t", gate, device, (E + S, f, d))
    _want("up_dense", up, device, (E + S, f, d), wdt)
    _want("down_dense", down, device, (E + S, d, f), wdt)
    if y is None:
        y = torch.empty((T, d), dtype=out_dtype or torch.float32, device=device)
    else:
        _want("y", y, device, (T, d))
    _want("residual", residual, device, (T, d), y.dtype)
    tr = None
    if trace:
        for name, t in trace.items():
            if name not in _TRACE_DTYPES:
                if t is None:
                    continue
                raise ValueError(f"layer_forward_few exports no {name}")
            shape = (T, k) if name[:4] == "topk" else (T, E) if name == "logits" else (E,)
            _want(name, t, device, shape, getattr(torch, _TRACE_DTYPES[name]))
        tr = C.byref(LayerTrace(**{name: _ptr(t) for name, t in trace.items() if t is not None}))
    ws, wp, wb = _workspace(torch, device, _size_of(OP_LAYER_FEW, T, d, f, E, k, S), ws)
    desc = LayerDesc(d=d, f=f, n_routed=E, n_shared=S, top_k=k, renormalize=int(bool(layer.renormalize)),
                     wdt=_dt(gate), router_w=_ptr(layer.router_w), rdt=_dt(layer.router_w),
                     router_bias=_ptr(layer.router_bias), gate_t=_ptr(gate), up_dense=_ptr(up),
                     down_dense=_ptr(down))
    _call(torch, device, "moe_layer_forward_few", lib().moe_layer_forward_few, C.byref(desc), _ptr(x),
          _dt(x), T, _ptr(residual), _ptr(y), _dt(y), tr, wp, wb)
    return y


@dataclass
class Linear:
    """A linear layer, y = act(x W^T + bias), or with w_gate
    y = act(x w_gate^T + bias_gate) * (x W^T + bias)."""
    w: "torch.Tensor"                           # [n][k] fp16/bf16
    bias: Optional["torch.Tensor"] = None       # [n] fp32
    w_gate: Optional["torch.Tensor"] = None     # [n][k]
    bias_gate: Optional["torch.Tensor"] = None  # [n] fp32
    act: str = "none"                           # a key of ACT

    @property
    def n(self):
        return self.w.shape[0]

    @property
    def k(self):
        return self.w.shape[1]

    def desc(self) -> LinearDesc:
        if self.act not in ACT:
            raise ValueError(f"act must be one of {sorted(ACT)}")
        return LinearDesc(self.w.shape[0], self.w.shape[1], _dt(self.w), _ptr(self.w), _ptr(self.bias),
                          _ptr(self.w_gate), _ptr(self.bias_gate), ACT[self.act])


def linear_forward(linear: Linear, x, *, residual=None, y=None, out_dtype=None, ws=None):
    """residual + the linear layer on x [T][k]; returns y [T][n].

    x, y and residual may be row-strided (contiguous rows; x's row stride a
    multiple of 8).  ``residual`` has y's type and may be y."""
    import torch
    if x.dim() != 2:
        raise ValueError("x must be [T][k]")
    device = x.device
    if device.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    w = linear.w
    T, (n, k) = x.shape[0], w.shape
    _want("x", x, device, (T, k))
    _want("w", w, device, (n, k))
    _want("bias", linear.bias, device, (n,), torch.float32)
    _want("w_gate", linear.w_gate, device, (n, k), w.dtype)
    _want("bias_gate", linear.bias_gate, device, (n,), torch.float32)
    if y is None:
        y = torch.empty((T, n), dtype=out_dtype or torch.float32, device=device)
    else:
        _want("y", y, device, (T, n))
    _want("residual", residual, device, (T, n), y.dtype)
    xp, xs = _rows("x", x, 8)
    yp, ys = _rows("y", y)
    rp, rs = _rows("residual", residual) if residual is not None else (None, 0)
    ws, wp, wb = _workspace(torch, device, _size_of(OP_LINEAR, T, k, n, 0, 0, 0), ws)
    _call(torch, device, "moe_linear_forward", lib().moe_linear_forward, C.byref(linear.desc()), xp,
          _dt(x), xs, T, rp, rs, yp, _dt(y), ys, wp, wb)
    return y


def linear_plan(T: int, k: int, n: int, gated: bool = False):
    """How linear_forward cuts a call of these sizes: ((tokens, weight rows) of a tile,
    parts of k), or (None, 0) where it streams the weights past the tokens."""
    return _plan(lib().moe_linear_plan, T, k, n, gated)


def linear_q8_plan(T: int, k: int, n: int, gated: bool = False):
    """linear_plan of linear_q8_forward."""
    return _plan(lib().moe_linear_q8_plan, T, k, n, gated)


def _plan(fn, T, k, n, gated):
    tokens, rows = C.c_int(), C.c_int()
    parts = fn(T, k, n, int(gated), C.byref(tokens), C.byref(rows))
    if parts < 0:
        raise ValueError(f"the linear layer does not take T = {T}, k = {k}, n = {n}")
    return ((tokens.value, rows.value) if parts else None), parts


@dataclass
class LinearQ8:
    """A linear layer on 8-bit weights: output j's weights are w_scale[j] w[j] (quantize_rows
    makes both from [n][k] weights), plain or gated as Linear."""
    w: "torch.Tensor"                            # [n][k] int8
    w_scale: "torch.Tensor"                      # [n] fp32
    bias: Optional["torch.Tensor"] = None        # [n] fp32
    w_gate: Optional["torch.Tensor"] = None      # [n][k] int8
    gate_scale: Optional["torch.Tensor"] = None  # [n] fp32
    bias_gate: Optional["torch.Tensor"] = None   # [n] fp32
    act: str = "none"                            # a key of ACT

    @property
    def n(self):
        return self.w.shape[0]

    @property
    def k(self):
        return self.w.shape[1]

    def desc(self) -> LinearQ8Desc:
        if self.act not in ACT:
            raise ValueError(f"act must be one of {sorted(ACT)}")
        return LinearQ8Desc(self.w.shape[0], self.w.shape[1], _ptr(self.w), _ptr(self.w_scale), _ptr(self.bias),
                            _ptr(self.w_gate), _ptr(self.gate_scale), _ptr(self.bias_gate), ACT[self.act])


_ROW_DT = {}


def _row_dt(t) -> int:
    """moe_dtype of a row operand: those of _dt, and codes."""
    dt = _ROW_DT.get(t.dtype)
    if dt is None:
        import torch
        _ROW_DT.update({torch.float16: MOE_F16, torch.bfloat16: MOE_BF16, torch.float32: MOE_F32, torch.int8: MOE_I8})
        dt = _ROW_DT.get(t.dtype)
        if dt is None:
            raise TypeError(f"unsupported dtype {t.dtype}")
    return dt


def linear_q8_forward(linear: LinearQ8, x, *, x_scale=None, residual=None, y=None, out_dtype=None, ws=None):
    """residual + the linear layer on x [T][k]: int8 codes with x_scale [T] (quantize_rows,
    norm_forward), or fp16, bf16 or fp32, which the call makes codes of; returns y [T][n].

    x, y and residual may be row-strided (contiguous rows; x's row stride a
    multiple of 16).  ``residual`` has y's type and may be y."""
    import torch
    if x.dim() != 2:
        raise ValueError("x must be [T][k]")
    device = x.device
    if device.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    w = linear.w
    T, (n, k) = x.shape[0], w.shape
    _want("x", x, device, (T, k))
    xdt = _row_dt(x)
    if (x_scale is None) == (xdt == MOE_I8):
        raise ValueError("x_scale comes with int8 codes and with nothing else")
    f32, sp, rp, rs = torch.float32, None, None, 0
    if x_scale is not None:
        _want("x_scale", x_scale, device, (T,), f32)
        sp = _ptr(x_scale)
    _want("w", w, device, (n, k), torch.int8)
    _want("w_scale", linear.w_scale, device, (n,), f32)
    if linear.bias is not None:
        _want("bias", linear.bias, device, (n,), f32)
    if (linear.w_gate is None) != (linear.gate_scale is None):
        raise ValueError("w_gate and gate_scale come together")
    if linear.w_gate is not None:
        _want("w_gate", linear.w_gate, device, (n, k), torch.int8)
        _want("gate_scale", linear.gate_scale, device, (n,), f32)
    if linear.bias_gate is not None:
        _want("bias_gate", linear.bias_gate, device, (n,), f32)
    if y is None:
        y = x.new_empty((T, n), dtype=out_dtype or f32)
        yp, ys = y.data_ptr(), n
    else:
        _want("y", y, device, (T, n))
        yp, ys = _rows("y", y)
    if residual is not None:
        _want("residual", residual, device, (T, n), y.dtype)
        rp, rs = _rows("residual", residual)
    xp, xs = _rows("x", x, 16)
    ws, wp, wb = _workspace(torch, device, _size_of(OP_LINEAR_Q8, T, k, n, xdt, 0, 0), ws)
    _call(torch, device, "moe_linear_q8_forward", lib().moe_linear_q8_forward, C.byref(linear.desc()), xp, xdt,
          xs, sp, T, rp, rs, yp, _row_dt(y), ys, wp, wb)
    return y


def quantize_rows(x, *, q=None, scale=None):
    """Rows of x [T][k] (fp16, bf16, fp32) as int8 codes q = round(127 x / max|x|), ties to
    even, with the scale max|x| / 127 of each row; returns (q [T][k], scale [T] fp32).
    Tokens for linear_q8_forward, or the weights [n][k] of a LinearQ8."""
    import torch
    if x.dim() != 2:
        raise ValueError("x must be [T][k]")
    device = x.device
    if device.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    T, k = x.shape
    if q is None:
        q = x.new_empty((T, k), dtype=torch.int8)
        qp, qs = q.data_ptr(), k
    else:
        _want("q", q, device, (T, k), torch.int8)
        qp, qs = _rows("q", q)
    if scale is None:
        scale = x.new_empty(T, dtype=torch.float32)
    else:
        _want("scale", scale, device, (T,), torch.float32)
    xp, xs = _rows("x", x)
    _call(torch, device, "moe_quantize_rows", lib().moe_quantize_rows, xp, _row_dt(x), xs, T, k, qp, qs, _ptr(scale))
    return q, scale


def dequantize_rows(q, scale, *, y=None, out_dtype=None):
    """The values q scale [T][k] that int8 codes [T][k] and their scales [T] stand for."""
    import torch
    if q.dim() != 2:
        raise ValueError("q must be [T][k]")
    device = q.device
    if device.type != "cuda":
        raise ValueError("q must be a GPU tensor")
    T, k = q.shape
    _want("q", q, device, (T, k), torch.int8)
    _want("scale", scale, device, (T,), torch.float32)
    if y is None:
        y = q.new_empty((T, k), dtype=out_dtype or torch.float32)
        yp, ys = y.data_ptr(), k
    else:
        _want("y", y, device, (T, k))
        yp, ys = _rows("y", y)
    qp, qs = _rows("q", q)
    _call(torch, device, "moe_dequantize_rows", lib().moe_dequantize_rows, qp, qs, _ptr(scale), T, k, yp, _row_dt(y), ys)
    return y


@dataclass
class Norm:
    """The norms between two blocks (norm_forward): RMS or layer norms of d channels."""
    d: int
    kind: str = "rms"                           # a key of NORM, for both norms
    eps: float = 1e-6
    w: Optional["torch.Tensor"] = None          # [d] of the norm before the next block (None: 1)
    b: Optional["torch.Tensor"] = None          # [d] (None: 0)
    post: bool = False                          # whether the block's output is normed too
    post_w: Optional["torch.Tensor"] = None     # [d]
    post_b: Optional["torch.Tensor"] = None     # [d]
    offset: bool = False                        # the weights are 1 + w, 1 + post_w
    residual_scale: float = 1.0
    block_scale: float = 1.0

    def desc(self) -> NormDesc:
        kind = NORM.get(self.kind)
        if kind is None:
            raise ValueError(f"kind must be one of {sorted(NORM)}")
        wdt, at = None, [None, None, None, None]
        for i, t in enumerate((self.w, self.b, self.post_w, self.post_b)):
            if t is not None:
                if wdt is None:
                    wdt = t.dtype
                    dt = _row_dt(t)
                elif t.dtype != wdt:
                    raise TypeError("the norms' weights and biases must have one dtype")
                at[i] = _ptr(t)
        return NormDesc(self.d, kind, self.eps, MOE_F32 if wdt is None else dt, at[0], at[1], int(bool(self.post)),
                        at[2], at[3], int(bool(self.offset)), self.residual_scale, self.block_scale)


def norm_forward(norm: Norm, residual, block=None, *, gate=None, y=None, out=None, out_dtype=None, out_scale=None):
    """Between two blocks: the first one's output, normed or not, gated and scaled, is added to
    the residual stream, and the norm before the second one is taken:
    v = residual_scale residual + block_scale (gate * Npost(block)), y = v, out = N(v).

    residual [T][d] or None (0); block [T][d] or None; gate, of the block's type, [T][d] or
    [d].  Returns (y, out, out_scale): y has the residual's type (without a residual the
    block's) and may be the residual, without a block it is written only if given; out has
    out_dtype, by default the block's or the residual's type, or as torch.int8 the codes of
    N(v) with out_scale [T].  y or out False: not wanted (None is returned)."""
    import torch
    x = residual if residual is not None else block
    if x is None:
        raise ValueError("norm_forward needs a residual or a block")
    shape, device = x.shape, x.device
    if len(shape) != 2:
        raise ValueError("residual and block must be [T][d]")
    if device.type != "cuda":
        raise ValueError("residual and block must be GPU tensors")
    T, d = shape
    if d != norm.d:
        raise ValueError(f"the rows have {d} columns, the norm d = {norm.d}")
    for t in (norm.w, norm.b, norm.post_w, norm.post_b):
        if t is not None and (t.device != device or t.shape != (d,)):
            _want("a norm's weight or bias", t, device, (d,))
    rp = bp = gp = yp = op = sp = None
    rs = bs = gs = ys = ns = bdt = odt = 0
    like = x
    xdt = _row_dt(x)
    if residual is not None:
        rp, rs = _rows("residual", residual)
    if block is not None:
        if block.device != device or block.shape != shape:
            _want("block", block, device, shape)
        bp, bs = _rows("block", block)
        bdt = _row_dt(block)
        like = block
    if gate is not None:
        if block is None:
            raise ValueError("a gate needs a block")
        _want("gate", gate, device, (d,) if gate.dim() == 1 else shape, block.dtype)
        gp, gs = (_ptr(gate), 0) if gate.dim() == 1 else _rows("gate", gate)
    if y is None:
        if block is not None:
            y = x.new_empty(shape)
            yp, ys = y.data_ptr(), d
    elif y is not False:
        _want("y", y, device, shape, x.dtype)
        yp, ys = _rows("y", y)
    if out is None:
        out = like.new_empty(shape) if out_dtype is None or out_dtype is like.dtype else like.new_empty(shape, dtype=out_dtype)
        op, ns = out.data_ptr(), d
    elif out is not False:
        _want("out", out, device, shape)
        op, ns = _rows("out", out)
    if op is not None:
        odt = _row_dt(out)
        if odt == MOE_I8 and out_scale is None:
            out_scale = x.new_empty(T, dtype=torch.float32)
    if out_scale is not None:
        _want("out_scale", out_scale, device, (T,), torch.float32)
        sp = _ptr(out_scale)
    _call(torch, device, "moe_norm_forward", lib().moe_norm_forward, C.byref(norm.desc()), T, rp, xdt, rs, bp, bdt, bs,
          gp, gs, yp, ys, op, odt, ns, sp)
    return None if y is False else y, None if out is False else out, out_scale


def calibrate_threshold(v, q: float, *, out=None, ws=None):
    """Threshold t = linear-interpolation q-quantile of |v| over all of the
    fp32 device tensor v, computed on the GPU; returns a one-element fp32
    device tensor."""
    import torch
    if v.dtype != torch.float32 or not v.is_contiguous():
        raise ValueError("v must be a contiguous fp32 tensor")
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=v.device)
    if ws is None:
        ws = new_workspace(workspace_size(OP_CALIBRATE, 1, 1), v.device)
    st = lib().moe_calibrate_threshold(_ptr(v), v.numel(), float(q), _ptr(out), _ptr(ws),
                                       ws.numel(), _stream())
    _check(st, "moe_calibrate_threshold")
    return out


def eamc_match(eamc, query, *, idx=None, dist=None, ws=None):
    """Cosine-distance nearest match of the int32 query [len] among the stored
    EAMs eamc [n][len] (both contiguous int32 device tensors, flattened L x E
    counts).  Returns (idx, dist): a one-element int32 tensor with the index
    (-1 when no stored EAM is valid) and, if ``dist`` was given or ``ws`` is
    None, the fp64 distances [n]."""
    import torch
    if eamc.dtype != torch.int32 or query.dtype != torch.int32:
        raise TypeError("eamc and query must be int32")
    if eamc.dim() != 2 or not eamc.is_contiguous() or not query.is_contiguous():
        raise ValueError("eamc must be a contiguous [n][len] tensor, query contiguous")
    n, ln = eamc.shape
    if query.numel() != ln:
        raise ValueError("query must have len entries")
    if idx is None:
        idx = torch.empty(1, dtype=torch.int32, device=eamc.device)
    if dist is None and ws is None:
        dist = torch.empty(n, dtype=torch.float64, device=eamc.device)
    st = lib().moe_eamc_match(_ptr(eamc), n, ln, _ptr(query), _ptr(idx), _ptr(dist), _ptr(ws),
                              0 if ws is None else ws.numel(), _stream())
    _check(st, "moe_eamc_match")
    return idx, dist


def pack_up_int2(w_up_t, *, up_q=None, up_sz=None):
    """INT2 group-64 quantisation of up weights [f][d] on the device."""
    import torch
    f, d = w_up_t.shape
    if up_q is None:
        up_q = torch.empty((f, d // 4), dtype=torch.uint8, device=w_up_t.device)
    if up_sz is None:
        up_sz = torch.empty((f, d // 64, 2), dtype=torch.int16, device=w_up_t.device)
    st = lib().moe_pack_up_int2(_ptr(w_up_t), _dt(w_up_t), d, f, _ptr(up_q), _ptr(up_sz),
                                _stream())
    _check(st, "moe_pack_up_int2")
    return up_q, up_sz


def pack_up_bits(w_up_t, bits: int, *, up_q=None, up_sz=None):
    """Group-64 quantisation of up weights [f][d] to 8, 4, 2 or 1 bits on the
    device; returns (up_q [f][d*bits/8] uint8, up_sz [f][d/64][2])."""
    import torch
    f, d = w_up_t.shape
    if up_q is None:
        up_q = torch.empty((f, d * bits // 8), dtype=torch.uint8, device=w_up_t.device)
    if up_sz is None:
        up_sz = torch.empty((f, d // 64, 2), dtype=torch.int16, device=w_up_t.device)
    st = lib().moe_pack_up_bits(_ptr(w_up_t), _dt(w_up_t), d, f, int(bits), _ptr(up_q),
                                _ptr(up_sz), _stream())
    _check(st, "moe_pack_up_bits")
    return up_q, up_sz


def materialize_up(up_q, up_sz, d: int, dtype, *, out=None):
    """Dense-path up weights [f][d] = rne(s (q - z)) in dtype (torch.bfloat16
    or torch.float16)."""
    import torch
    f = up_q.shape[0]
    if out is None:
        out = torch.empty((f, d), dtype=dtype, device=up_q.device)
    st = lib().moe_materialize_up(_ptr(up_q), _ptr(up_sz), d, f, _dt(out), _ptr(out), _stream())
    _check(st, "moe_materialize_up")
    return out


def transpose_down(down, *, out=None):
    """Dense-path down weights: [n][d][f] (or [d][f]) = the transpose of each
    expert's down [f][d]."""
    import torch
    squeeze = down.dim() == 2
    dn = down.unsqueeze(0) if squeeze else down
    n, f, d = dn.shape
    if out is None:
        out = torch.empty((n, d, f), dtype=down.dtype, device=down.device)
    st = lib().moe_transpose_down(_ptr(dn), n, d, f, _ptr(out), _stream())
    _check(st, "moe_transpose_down")
    return out[0] if squeeze else out


def materialize_up_bf16(up_q, up_sz, d: int, *, out=None):
    """bf16 up weights [f][d] = bf16_rne(s (q - z)) for the dense path."""
    import torch
    f = up_q.shape[0]
    if out is None:
        out = torch.empty((f, d), dtype=torch.bfloat16, device=up_q.device)
    st = lib().moe_materialize_up_bf16(_ptr(up_q), _ptr(up_sz), d, f, _ptr(out), _stream())
    _check(st, "moe_materialize_up_bf16")
    return out
