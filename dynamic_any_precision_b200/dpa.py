"""Thin Python binding of the C ABI in include/dpa.h (argument marshalling only).

Device buffers are torch CUDA tensors (PyTorch provides memory and streams); every
computation runs in the CUDA library lib/libdpa_b200.so. There is no CPU fallback: if the
library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
# the in-tree build; DPA_LIB may name another build of the same library (e.g. a debug build)
LIB_PATH = os.environ.get("DPA_LIB") or os.path.join(_PKG, "lib", "libdpa_b200.so")

DPA_OK = 0
STATUS_NAMES = {0: "DPA_OK", 1: "DPA_ERR_INVALID_ARG", 2: "DPA_ERR_UNSUPPORTED", 3: "DPA_ERR_WORKSPACE",
                4: "DPA_ERR_CUDA", 5: "DPA_ERR_DEVICE_TIMEOUT", 6: "DPA_ERR_DEVICE_INVALID_INPUT"}
FMT_UNIFORM, FMT_BCQ = 0, 1
MAT_GATE, MAT_UP, MAT_DOWN = 0, 1, 2


class DpaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")
        self.status = status


class LayerDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("hidden", "inter", "n_experts", "top_k", "n_shared", "format", "bits", "kmin", "kmax",
                 "group", "norm_topk")]


class Sizes(ctypes.Structure):
    _fields_ = [("planes_bytes", ctypes.c_uint64), ("meta_bytes", ctypes.c_uint64),
                ("rtable_bytes", ctypes.c_uint64), ("planes_per_expert", ctypes.c_uint64),
                ("meta_per_expert", ctypes.c_uint64), ("planes_matrix_offset", ctypes.c_uint64 * 3),
                ("meta_matrix_offset", ctypes.c_uint64 * 3)]


class LayerWeights(ctypes.Structure):
    _fields_ = [("planes", ctypes.c_void_p), ("meta", ctypes.c_void_p), ("rtable", ctypes.c_void_p),
                ("w_router", ctypes.c_void_p), ("shared_gate", ctypes.c_void_p),
                ("shared_up", ctypes.c_void_p), ("shared_down", ctypes.c_void_p),
                ("expert_width", ctypes.c_void_p), ("expert_offsets", ctypes.c_void_p)]


class LinearDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("rows", "in_features", "out_features", "dtype", "out_dtype", "act", "residual_dtype")]


class Aux(ctypes.Structure):
    _fields_ = [("topk_idx", ctypes.c_void_p), ("topk_gate", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("lambda_", ctypes.c_void_p), ("pair_out", ctypes.c_void_p),
                ("events", ctypes.c_void_p * 7), ("expert_path", ctypes.c_int32),
                ("alloc_policy", ctypes.c_int32), ("threshold", ctypes.c_void_p), ("expert_k", ctypes.c_void_p)]

PATH_AUTO, PATH_GEMV, PATH_TC = 0, 1, 2
ALLOC_LAGRANGE, ALLOC_UNIFORM, ALLOC_THRESHOLD, ALLOC_EXPERT_TABLE = 0, 1, 2, 3
DTYPE_BF16, DTYPE_FP16, DTYPE_FP32, DTYPE_FP64 = 0, 1, 2, 3
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3, 4
ACTS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH, "silu": ACT_SILU}
LINEAR_WORKSPACE_BYTES = 256


EXPORTED = ("dpa_encoded_sizes", "dpa_encode", "dpa_export_codes", "dpa_export_meta", "dpa_route",
            "dpa_allocate", "dpa_allocate_ex", "dpa_calibrate_threshold", "dpa_forward_workspace_size",
            "dpa_moe_forward", "dpa_device_status", "dpa_status_string", "dpa_version", "dpa_residual_rmsnorm",
            "dpa_debug_timeout_probe", "dpa_distortion_tensor", "dpa_profile_prefill", "dpa_solve_expert_rates",
            "dpa_stream_prefixes", "dpa_solve_stored_widths", "dpa_compact_sizes", "dpa_compact_layer",
            "dpa_sort_workspace_size", "dpa_sort_pairs", "dpa_permute_rows", "dpa_unpermute_rows",
            "dpa_unpermute_rows_backward", "dpa_linear", "dpa_grouped_linear")

_lib = None


def lib() -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                           "(run `python -m dynamic_any_precision_b200.build`)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    P = ctypes.POINTER
    L.dpa_encoded_sizes.argtypes = [P(LayerDesc), P(Sizes)]
    L.dpa_encode.argtypes = [P(LayerDesc), i32, i32, vp, vp, vp, vp, vp, vp, i32]
    L.dpa_export_codes.argtypes = [P(LayerDesc), vp, i32, i32, vp]
    L.dpa_export_meta.argtypes = [P(LayerDesc), vp, i32, i32, vp, vp]
    L.dpa_route.argtypes = [P(LayerDesc), vp, i32, vp, vp, vp, vp, vp, sz, vp]
    L.dpa_allocate.argtypes = [P(LayerDesc), vp, vp, vp, i32, vp, vp, vp, vp, sz, vp]
    L.dpa_allocate_ex.argtypes = [P(LayerDesc), i32, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.dpa_distortion_tensor.argtypes = [P(LayerDesc), i32, i32, vp, vp, vp, vp, vp, i32]
    L.dpa_profile_prefill.argtypes = [P(LayerDesc), vp, i32, vp, vp, vp, vp, sz, vp]
    L.dpa_solve_expert_rates.argtypes = [P(LayerDesc), vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.dpa_calibrate_threshold.argtypes = [P(LayerDesc), vp, i32, vp, vp, vp, sz, vp]
    L.dpa_forward_workspace_size.argtypes = [P(LayerDesc), i32]
    L.dpa_forward_workspace_size.restype = sz
    L.dpa_moe_forward.argtypes = [P(LayerDesc), P(LayerWeights), vp, i32, vp, vp, P(Aux), vp, sz, vp]
    L.dpa_device_status.argtypes = [vp, vp]
    L.dpa_debug_timeout_probe.argtypes = [vp, sz, i32, ctypes.c_uint64, vp]
    L.dpa_stream_prefixes.argtypes = [P(LayerDesc), vp, vp, vp, vp, i32, vp, vp, P(ctypes.c_uint64), vp]
    L.dpa_residual_rmsnorm.argtypes = [vp, vp, i32, i32, vp, vp]
    L.dpa_solve_stored_widths.argtypes = [P(LayerDesc), vp, vp, ctypes.c_int64, vp]
    L.dpa_compact_sizes.argtypes = [P(LayerDesc), vp, P(ctypes.c_uint64), P(ctypes.c_uint64)]
    L.dpa_compact_layer.argtypes = [P(LayerDesc), vp, vp, vp, vp, vp, vp]
    L.dpa_sort_workspace_size.argtypes = [i32, i32]
    L.dpa_sort_workspace_size.restype = sz
    L.dpa_sort_pairs.argtypes = [vp, i32, i32, vp, vp, vp, vp, sz, vp]
    L.dpa_permute_rows.argtypes = [i32, vp, vp, i32, i32, i32, vp, vp]
    L.dpa_unpermute_rows.argtypes = [i32, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, vp, vp]
    L.dpa_unpermute_rows_backward.argtypes = [i32, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp]
    L.dpa_linear.argtypes = [P(LinearDesc), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.dpa_grouped_linear.argtypes = [P(LinearDesc), i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.dpa_status_string.argtypes = [i32]
    L.dpa_status_string.restype = ctypes.c_char_p
    L.dpa_version.argtypes = []
    for name in EXPORTED:
        if name not in ("dpa_forward_workspace_size", "dpa_sort_workspace_size", "dpa_status_string", "dpa_version"):
            getattr(L, name).restype = i32
    L.dpa_version.restype = i32
    _lib = L
    return L


def _check(st: int, where: str):
    if st != DPA_OK:
        raise DpaError(st, where)


def make_desc(shape) -> LayerDesc:
    """Descriptor from a workloads.LayerShape (or any object with the same fields)."""
    return LayerDesc(shape.hidden, shape.inter, shape.n_experts, shape.top_k, shape.n_shared, shape.fmt,
                     shape.bits, shape.kmin, shape.kmax, shape.group, shape.norm_topk)


def encoded_sizes(desc: LayerDesc) -> Sizes:
    s = Sizes()
    _check(lib().dpa_encoded_sizes(ctypes.byref(desc), ctypes.byref(s)), "dpa_encoded_sizes")
    return s


def _ptr(a: np.ndarray) -> int:
    return a.ctypes.data


def encode(desc: LayerDesc, w_gate: np.ndarray, w_up: np.ndarray, w_down: np.ndarray, e_begin: int = 0,
           out: Optional[Tuple[np.ndarray, np.ndarray, np.ndarray]] = None, n_threads: int = 0):
    """Host encoder. w_* hold experts [e_begin, e_begin + n) as contiguous fp32 arrays.
    Returns (planes uint8, meta uint8, rtable fp64 [E][B]) for the whole layer (only the
    given experts' parts are written; pass `out` to fill buffers from earlier calls)."""
    s = encoded_sizes(desc)
    if out is None:
        planes = np.zeros(s.planes_bytes, np.uint8)
        meta = np.zeros(s.meta_bytes, np.uint8)
        rtable = np.zeros((desc.n_experts, desc.bits), np.float64)
    else:
        planes, meta, rtable = out
    wg = np.ascontiguousarray(w_gate, np.float32)
    wu = np.ascontiguousarray(w_up, np.float32)
    wd = np.ascontiguousarray(w_down, np.float32)
    n = wg.shape[0] if wg.ndim == 3 else 1
    _check(lib().dpa_encode(ctypes.byref(desc), e_begin, n, _ptr(wg), _ptr(wu), _ptr(wd), _ptr(planes), _ptr(meta),
                            _ptr(rtable), n_threads), "dpa_encode")
    return planes, meta, rtable


def export_codes(desc: LayerDesc, planes: np.ndarray, expert: int, matrix: int) -> np.ndarray:
    R = desc.hidden if matrix == MAT_DOWN else desc.inter
    C = desc.inter if matrix == MAT_DOWN else desc.hidden
    out = np.empty((R, C), np.uint8)
    _check(lib().dpa_export_codes(ctypes.byref(desc), _ptr(planes), expert, matrix, _ptr(out)), "dpa_export_codes")
    return out


def export_meta(desc: LayerDesc, meta: np.ndarray, expert: int, matrix: int):
    R = desc.hidden if matrix == MAT_DOWN else desc.inter
    C = desc.inter if matrix == MAT_DOWN else desc.hidden
    ng = C // desc.group
    if desc.format == FMT_UNIFORM:
        s = np.empty((R, ng), np.float32)
        z = np.empty((R, ng), np.float32)
        _check(lib().dpa_export_meta(ctypes.byref(desc), _ptr(meta), expert, matrix, _ptr(s), _ptr(z)),
               "dpa_export_meta")
        return s, z
    al = np.empty((desc.bits, R, ng), np.float32)
    _check(lib().dpa_export_meta(ctypes.byref(desc), _ptr(meta), expert, matrix, _ptr(al), None), "dpa_export_meta")
    return al, None


# ----------------------------------------------------------------------------- device calls

def _stream(stream=None) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _dptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def workspace_size(desc: LayerDesc, max_tokens: int) -> int:
    n = lib().dpa_forward_workspace_size(ctypes.byref(desc), max_tokens)
    if n == 0:
        raise DpaError(1, "dpa_forward_workspace_size")
    return n


def new_workspace(desc: LayerDesc, max_tokens: int, device=None):
    """Zero-filled workspace (the library requires it zeroed once before first use)."""
    import torch
    return torch.zeros(workspace_size(desc, max_tokens), dtype=torch.uint8, device=device or "cuda")


def route(desc: LayerDesc, x, w_router, ws, logits=None, stream=None):
    """x: CUDA uint16/bf16 [T][H]; w_router: [E][H]. Returns (idx int32 [T][K], gate fp64 [T][K])."""
    import torch
    T = x.shape[0]
    idx = torch.empty((T, desc.top_k), dtype=torch.int32, device=x.device)
    gate = torch.empty((T, desc.top_k), dtype=torch.float64, device=x.device)
    _check(lib().dpa_route(ctypes.byref(desc), _dptr(x), T, _dptr(w_router), _dptr(idx), _dptr(gate),
                           _dptr(logits), _dptr(ws), ws.numel(), _stream(stream)), "dpa_route")
    return idx, gate


def allocate(desc: LayerDesc, rtable, idx, gate, target, ws, stream=None, policy: int = ALLOC_LAGRANGE,
             threshold=None, expert_k=None):
    """target: CUDA fp64 scalar tensor (None for the threshold and table policies); threshold:
    CUDA fp64 scalar tensor (threshold policy); expert_k: CUDA uint8 [E] (table policy).
    Returns (k uint8 [T][K], lambda fp64 [1])."""
    import torch
    T = idx.shape[0]
    k = torch.empty((T, desc.top_k), dtype=torch.uint8, device=idx.device)
    lam = torch.empty(1, dtype=torch.float64, device=idx.device)
    if policy == ALLOC_LAGRANGE:
        _check(lib().dpa_allocate(ctypes.byref(desc), _dptr(rtable), _dptr(idx), _dptr(gate), T, _dptr(target),
                                  _dptr(k), _dptr(lam), _dptr(ws), ws.numel(), _stream(stream)), "dpa_allocate")
    else:
        _check(lib().dpa_allocate_ex(ctypes.byref(desc), policy, _dptr(rtable), _dptr(idx), _dptr(gate), T,
                                     _dptr(target), _dptr(threshold), _dptr(expert_k), _dptr(k), _dptr(lam),
                                     _dptr(ws), ws.numel(), _stream(stream)), "dpa_allocate_ex")
    return k, lam


def distortion_tensor(desc: LayerDesc, w_gate: np.ndarray, w_up: np.ndarray, planes: np.ndarray, meta: np.ndarray,
                      e_begin: int = 0, out: Optional[np.ndarray] = None, n_threads: int = 0) -> np.ndarray:
    """Host distortion tensor [E][B][H] fp64 for experts [e_begin, e_begin + n) of the layer."""
    T = np.zeros((desc.n_experts, desc.bits, desc.hidden), np.float64) if out is None else out
    wg = np.ascontiguousarray(w_gate, np.float32)
    wu = np.ascontiguousarray(w_up, np.float32)
    n = wg.shape[0] if wg.ndim == 3 else 1
    _check(lib().dpa_distortion_tensor(ctypes.byref(desc), e_begin, n, _ptr(wg), _ptr(wu), _ptr(planes), _ptr(meta),
                                       _ptr(T), n_threads), "dpa_distortion_tensor")
    return T


def profile_prefill(desc: LayerDesc, x, idx, ws, stream=None):
    """x: CUDA bf16 bits [T][H]; idx: CUDA int32 [T][K]. Returns (m fp64 [H], counts int32 [E])."""
    import torch
    m = torch.empty(desc.hidden, dtype=torch.float64, device=x.device)
    counts = torch.empty(desc.n_experts, dtype=torch.int32, device=x.device)
    _check(lib().dpa_profile_prefill(ctypes.byref(desc), _dptr(x), x.shape[0], _dptr(idx), _dptr(m), _dptr(counts),
                                     _dptr(ws), ws.numel(), _stream(stream)), "dpa_profile_prefill")
    return m, counts


def solve_expert_rates(desc: LayerDesc, tdist, m, counts, target, ws, stream=None):
    """tdist: CUDA fp64 [E][B][H]. Returns (k_table uint8 [E], lambda fp64 [1])."""
    import torch
    kt = torch.empty(desc.n_experts, dtype=torch.uint8, device=m.device)
    lam = torch.empty(1, dtype=torch.float64, device=m.device)
    _check(lib().dpa_solve_expert_rates(ctypes.byref(desc), _dptr(tdist), _dptr(m), _dptr(counts), _dptr(target),
                                        _dptr(kt), _dptr(lam), _dptr(ws), ws.numel(), _stream(stream)),
           "dpa_solve_expert_rates")
    return kt, lam


def calibrate_threshold(desc: LayerDesc, scores, target, ws, stream=None):
    """scores: CUDA fp64 tensor (any shape) of calibration routing scores; target: CUDA fp64
    scalar tensor. Returns the threshold as a CUDA fp64 [1] tensor."""
    import torch
    tau = torch.empty(1, dtype=torch.float64, device=scores.device)
    _check(lib().dpa_calibrate_threshold(ctypes.byref(desc), _dptr(scores), scores.numel(), _dptr(target), _dptr(tau),
                                         _dptr(ws), ws.numel(), _stream(stream)), "dpa_calibrate_threshold")
    return tau


class DeviceLayer:
    """Encoded layer resident in device memory (torch tensors) plus its C weight struct."""

    def __init__(self, desc: LayerDesc, planes, meta, rtable, w_router, shared=None, widths=None, offsets=None):
        """widths (uint8 [E]) and offsets (uint64 [E][2] as int64) on the device: a compact layer
        of per-expert stored widths (dpa_compact_layer); both None: the full layout."""
        self.desc = desc
        self.planes, self.meta, self.rtable, self.w_router = planes, meta, rtable, w_router
        self.shared = shared
        self.widths, self.offsets = widths, offsets
        sg, su, sd = shared if shared is not None else (None, None, None)
        self.weights = LayerWeights(_dptr(planes), _dptr(meta), _dptr(rtable), _dptr(w_router), _dptr(sg),
                                    _dptr(su), _dptr(sd), _dptr(widths), _dptr(offsets))

    @classmethod
    def from_host(cls, desc: LayerDesc, planes: np.ndarray, meta: np.ndarray, rtable: np.ndarray,
                  w_router_bits: np.ndarray, shared_bits=None, device="cuda"):
        import torch

        def dev(a):
            return torch.from_numpy(np.ascontiguousarray(a)).to(device)
        sh = None
        if shared_bits is not None:
            sh = tuple(dev(s.view(np.int16)) for s in shared_bits)
        return cls(desc, dev(planes), dev(meta), dev(rtable), dev(w_router_bits.view(np.int16)), sh)


def moe_forward(layer: DeviceLayer, x, target, ws, y=None, aux: Optional[dict] = None, stream=None):
    """One MoE layer. x: CUDA int16/bf16 bits [T][H]; target: CUDA fp64 scalar tensor.
    aux: optional dict of preallocated CUDA tensors with keys topk_idx, topk_gate, k, lambda,
    pair_out, "events": up to 7 torch.cuda.Event(enable_timing=True) recorded at the
    stage boundaries, "expert_path" (PATH_AUTO, PATH_GEMV or PATH_TC), "alloc_policy"
    (ALLOC_LAGRANGE, ALLOC_UNIFORM or ALLOC_THRESHOLD) and "threshold" (CUDA fp64 scalar).
    Returns y (int16 bf16 bits [T][H])."""
    import torch
    T = x.shape[0]
    if y is None:
        y = torch.empty((T, layer.desc.hidden), dtype=torch.int16, device=x.device)
    aux_s = None
    if aux:
        aux_s = Aux(_dptr(aux.get("topk_idx")), _dptr(aux.get("topk_gate")), _dptr(aux.get("k")),
                    _dptr(aux.get("lambda")), _dptr(aux.get("pair_out")))
        for i, ev in enumerate(aux.get("events") or ()):
            if ev is not None:
                if not ev.cuda_event:
                    raise ValueError("record a torch.cuda.Event once before passing it (lazy creation)")
                aux_s.events[i] = ev.cuda_event
        aux_s.expert_path = int(aux.get("expert_path", PATH_AUTO))
        aux_s.alloc_policy = int(aux.get("alloc_policy", ALLOC_LAGRANGE))
        aux_s.threshold = _dptr(aux.get("threshold"))
        aux_s.expert_k = _dptr(aux.get("expert_k"))
    _check(lib().dpa_moe_forward(ctypes.byref(layer.desc), ctypes.byref(layer.weights), _dptr(x), T, _dptr(target),
                                 _dptr(y), ctypes.byref(aux_s) if aux_s is not None else None, _dptr(ws), ws.numel(),
                                 _stream(stream)), "dpa_moe_forward")
    return y


def residual_rmsnorm(h, x, y=None, stream=None):
    """Stack glue: h += y (if given), x = bf16(RMSNorm(h)). h fp32 [T][H] (in place),
    x and y bf16 bits [T][H] (int16 tensors)."""
    T, H = h.shape
    _check(lib().dpa_residual_rmsnorm(_dptr(y), _dptr(h), T, H, _dptr(x), _stream(stream)), "dpa_residual_rmsnorm")
    return x


# ------------------------------------------------------------- dense experts: rows and products
# These calls record no autograd history: their results never require gradients, whatever the inputs do.
# The row calls' gradients are calls of their own; the products have none.

_DTYPES = _FLOATS = None
_current_device = _raw_stream = _empty_like = _empty_strided = None


def _torch_tables():
    """Element types and the current device and stream, looked up once (torch is imported late).
    int16 and uint16 tensors hold bf16 bit patterns."""
    global _DTYPES, _FLOATS, _current_device, _raw_stream, _empty_like, _empty_strided
    import torch
    _FLOATS = {torch.bfloat16: DTYPE_BF16, torch.int16: DTYPE_BF16, torch.uint16: DTYPE_BF16,
               torch.float16: DTYPE_FP16, torch.float32: DTYPE_FP32, torch.float64: DTYPE_FP64}
    _DTYPES = {**_FLOATS, torch.int32: "int32", torch.uint8: "uint8"}
    _current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _empty_like, _empty_strided = torch.empty_like, torch.empty_strided


def _device(t) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError("expected a CUDA tensor")
    if _DTYPES is None:
        _torch_tables()
    return dev


def _float_type(t) -> int:
    """DTYPE_* of a tensor of floating-point values."""
    code = _FLOATS.get(t.dtype)
    if code is None:
        raise ValueError(f"unsupported element type {t.dtype}")
    return code


def _arg(t, name: str, shape, code, dev: int) -> int:
    """Pointer of a tensor argument, after checking its shape, element type (DTYPE_*, "int32" or
    "uint8"), device index and layout."""
    if t.shape == shape and _DTYPES.get(t.dtype) == code and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if _DTYPES.get(t.dtype) != code:
        raise ValueError(f"{name}: unexpected element type {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on cuda:{dev}, got {t.device}")
    raise ValueError(f"{name}: expected a contiguous tensor")


def _own(t, name: str) -> int:
    """Pointer of the tensor that the call's sizes, type and device are taken from, or that the call
    has made itself."""
    if t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: expected a contiguous tensor")


def _workspace(ws, dev: int) -> int:
    if _DTYPES.get(ws.dtype) == "uint8" and ws.get_device() == dev and ws.is_contiguous():
        return ws.data_ptr()
    return _arg(ws, "ws", ws.shape, "uint8", dev)   # names what is wrong


def _call(fn, where: str, dev: int, stream, *args):
    """Run a device call on `dev`, on the given stream or that device's current one."""
    raw = _raw_stream(dev) if stream is None else stream.cuda_stream
    if _current_device() == dev:
        st = fn(*args, raw)
    else:
        import torch
        with torch.cuda.device(dev):
            st = fn(*args, raw)
    if st != DPA_OK:
        raise DpaError(st, where)


def _new(like, shape, dtype, stream):
    """A new tensor on `like`'s device, taken from the memory of the stream that the call runs on.
    shape: (n,) or (n, m), with its strides given (empty_strided takes 1.4 us of host time, new_empty
    2.2 to 3.5)."""
    strides = (1,) if len(shape) == 1 else (shape[1], 1)
    if stream is None:
        return _empty_strided(shape, strides, dtype=dtype, device=like.device)
    import torch
    with torch.cuda.stream(stream):
        return _empty_strided(shape, strides, dtype=dtype, device=like.device)


def _like(t, stream):
    """_new of t's own shape and type."""
    if stream is None:
        return _empty_like(t)
    import torch
    with torch.cuda.stream(stream):
        return _empty_like(t)


# Sizes go to the library as 32-bit integers, and ctypes passes the low 32 bits of a larger one: the calls
# below refuse those (DPA_ERR_UNSUPPORTED) before it could take them for small sizes.

def sort_workspace_size(n_pairs: int, n_experts: int) -> int:
    n = 0 if (n_pairs | n_experts) >> 31 else lib().dpa_sort_workspace_size(n_pairs, n_experts)
    if n == 0:
        raise DpaError(1, "dpa_sort_workspace_size")
    return n


def new_sort_workspace(n_pairs: int, n_experts: int, device=None):
    """Zero-filled workspace for sort_pairs of up to n_pairs pairs (serves linear and
    grouped_linear too)."""
    import torch
    return torch.zeros(sort_workspace_size(n_pairs, n_experts), dtype=torch.uint8, device=device or "cuda")


def new_linear_workspace(device=None):
    """Zero-filled workspace for linear and grouped_linear: it holds the device error flag only
    (device_status reads it), so any workspace of the library serves as well."""
    import torch
    return torch.zeros(LINEAR_WORKSPACE_BYTES, dtype=torch.uint8, device=device or "cuda")


def sort_pairs(idx, n_experts: int, ws, pos=None, order=None, offsets=None, stream=None):
    """Stable sort of routed pairs by expert. idx: CUDA int32, any shape (one expert id per pair;
    ids outside [0, n_experts) are not routed). Returns (pos in idx's shape, order [P], offsets
    [n_experts + 1]), int32: the place of each pair (-1 if not routed), the pair at each place
    (unrouted ones last), the places before each expert."""
    dev, P = _device(idx), idx.numel()
    if (P | n_experts) >> 31:
        raise DpaError(1 if n_experts < 0 else 2, "dpa_sort_pairs")
    ip = _arg(idx, "idx", idx.shape, "int32", dev)
    if pos is None:
        pos = _like(idx, stream)
        pp = pos.data_ptr()
    else:
        pp = _arg(pos, "pos", idx.shape, "int32", dev)
    if order is None:
        order = _new(idx, (P,), idx.dtype, stream)
        op = order.data_ptr()
    else:
        op = _arg(order, "order", (P,), "int32", dev)
    if offsets is None:
        offsets = _new(idx, (n_experts + 1,), idx.dtype, stream)
        fp = offsets.data_ptr()
    else:
        fp = _arg(offsets, "offsets", (n_experts + 1,), "int32", dev)
    _call(lib().dpa_sort_pairs, "dpa_sort_pairs", dev, stream, ip, P, n_experts, pp, op, fp, _workspace(ws, dev),
          ws.numel())
    return pos, order, offsets


def permute_rows(x, pos, out=None, stream=None):
    """out[pos[t][k]] = x[t]. x: [T][H] bf16 (or int16 bits), fp16 or fp32; pos: int32 [T][K] from
    sort_pairs. Returns out [T*K][H]; rows that no pair takes are left as they were (with out=None:
    uninitialised)."""
    dev, code = _device(x), _float_type(x)
    (T, H), K = x.shape, pos.shape[-1]
    if (T | K | H) >> 31:
        raise DpaError(2, "dpa_permute_rows")
    xp, pp = _own(x, "x"), _arg(pos, "pos", (T, K), "int32", dev)
    if out is None:
        out = _new(x, (T * K, H), x.dtype, stream)
        yp = out.data_ptr()
    else:
        yp = _arg(out, "out", (T * K, H), code, dev)
    _call(lib().dpa_permute_rows, "dpa_permute_rows", dev, stream, code, xp, pp, T, K, H, yp)
    return out


def permute_rows_backward(dout, pos, dx=None, stream=None):
    """Gradient of permute_rows: dx[t] = sum_k dout[pos[t][k]] (fp32 sums, rounded once)."""
    return unpermute_rows(dout, pos, None, out=dx, stream=stream)


def _out(out, shape, like, residual, out_dtype, stream):
    """The output tensor of a call: the given one, or a new one of out_dtype (default: the
    residual's type, else `like`'s)."""
    if out is None:
        if residual is not None and residual.shape == shape and out_dtype in (None, residual.dtype):
            return _like(residual, stream)
        return _new(like, shape, out_dtype or (like if residual is None else residual).dtype, stream)
    if out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out: unexpected element type {out.dtype}")
    return out


def unpermute_rows(z, pos, weights=None, residual=None, out=None, out_dtype=None, stream=None):
    """y[t] = residual[t] + sum_k weights[t][k] * z[pos[t][k]]. z: [T*K][H]; pos: int32 [T][K];
    weights: fp32 or fp64 [T][K] (None: all 1); residual: [T][H] of y's type or fp32, may be `out`.
    y has out_dtype (default: residual's, else z's): z's own type, or one of the two is fp32."""
    dev, (T, K), H = _device(z), pos.shape, z.shape[-1]
    if (T | K | H) >> 31:
        raise DpaError(2, "dpa_unpermute_rows")
    given, out = out is not None, _out(out, (T, H), z, residual, out_dtype, stream)
    code, zcode, wcode = _float_type(out), _float_type(z), _real(weights)
    rcode = code if residual is None else _float_type(residual)
    _call(lib().dpa_unpermute_rows, "dpa_unpermute_rows", dev, stream, zcode,
          _arg(z, "z", (T * K, H), zcode, dev), _arg(pos, "pos", (T, K), "int32", dev),
          None if weights is None else _arg(weights, "weights", (T, K), wcode, dev), wcode,
          None if residual is None else _arg(residual, "residual", (T, H), rcode, dev), rcode, code, T, K, H,
          _arg(out, "out", (T, H), code, dev) if given else out.data_ptr())
    return out


def _real(weights) -> int:
    """DTYPE_* of gate weights (fp32 or fp64), -1 without weights."""
    if weights is None:
        return -1
    code = _FLOATS.get(weights.dtype)
    if code not in (DTYPE_FP32, DTYPE_FP64):
        raise ValueError(f"weights: expected fp32 or fp64, got {weights.dtype}")
    return code


def unpermute_rows_backward(dy, z, pos, weights, dz=None, dweights=None, stream=None):
    """Gradients of unpermute_rows: (dz [T*K][H] in z's type, dweights fp32 [T][K]). dy: [T][H] of
    z's type; dz may be z. Rows of dz that no pair takes are left as they were (with dz=None: uninitialised);
    pairs that are not routed get dweights 0. The residual's gradient is dy itself."""
    dev, (T, K), H = _device(z), pos.shape, z.shape[-1]
    if (T | K | H) >> 31:
        raise DpaError(2, "dpa_unpermute_rows_backward")
    code, wcode = _float_type(z), _real(weights)
    if weights is None:
        raise ValueError("weights: expected a tensor")
    zp = _arg(z, "z", (T * K, H), code, dev)
    if dz is None:
        dz = _like(z, stream)
        dzp = dz.data_ptr()
    else:
        dzp = _arg(dz, "dz", (T * K, H), code, dev)
    if dweights is None:
        import torch
        dweights = _new(z, (T, K), torch.float32, stream)
        dwp = dweights.data_ptr()
    else:
        dwp = _arg(dweights, "dweights", (T, K), DTYPE_FP32, dev)
    _call(lib().dpa_unpermute_rows_backward, "dpa_unpermute_rows_backward", dev, stream, code,
          _arg(dy, "dy", (T, H), code, dev), zp,
          _arg(pos, "pos", (T, K), "int32", dev), _arg(weights, "weights", (T, K), wcode, dev), wcode, T, K, H,
          dzp, dwp)
    return dz, dweights


def _product(fn, where, x, w, lead, groups, ws, bias, act, w_mul, bias_mul, residual, out, out_dtype, stream):
    """linear and grouped_linear: `lead` is () or (n_groups,), `groups` the group arguments of the
    call: () or (n_groups, offsets)."""
    dev, (rows, K), N = _device(x), x.shape, w.shape[-2]
    if (rows | K | N | (lead[0] if lead else 0)) >> 31:
        raise DpaError(2, where)
    wide, flat, rect = lead + (N, K), lead + (N,), (rows, N)
    given, out = out is not None, _out(out, rect, x, residual, out_dtype, stream)
    code, ocode = _float_type(x), _float_type(out)
    rcode = ocode if residual is None else _float_type(residual)
    if act not in ACTS:
        raise ValueError(f"act: expected one of {', '.join(ACTS)}, got {act!r}")
    xp = _own(x, "x")
    if groups:
        groups = (groups[0], xp, _arg(groups[1], "offsets", (groups[0] + 1,), "int32", dev))
    else:
        groups = (xp,)
    _call(fn, where, dev, stream, LinearDesc(rows, K, N, code, ocode, ACTS[act], rcode), *groups,
          _arg(w, "w", wide, code, dev), None if bias is None else _arg(bias, "bias", flat, code, dev),
          None if w_mul is None else _arg(w_mul, "w_mul", wide, code, dev),
          None if bias_mul is None else _arg(bias_mul, "bias_mul", flat, code, dev),
          None if residual is None else _arg(residual, "residual", rect, rcode, dev),
          _arg(out, "out", rect, ocode, dev) if given else out.data_ptr(), _workspace(ws, dev), ws.numel())
    return out


def linear(x, w, ws, bias=None, act="none", w_mul=None, bias_mul=None, residual=None, out=None, out_dtype=None,
           stream=None):
    """out = act(x w^T + bias) [* (x w_mul^T + bias_mul)] [+ residual]. x: [M][K] bf16 (or int16
    bits) or fp16, K a multiple of 8; w, w_mul: [N][K]; bias, bias_mul: [N], all of x's type; out:
    [M][N] in x's type or fp32 (out_dtype; default: residual's, else x's); residual: [M][N] of
    out's type or fp32, may be `out`. act: "none", "relu", "gelu", "gelu_tanh" or "silu". ws:
    new_linear_workspace or any other workspace; it receives the device error flag."""
    return _product(lib().dpa_linear, "dpa_linear", x, w, (), (), ws, bias, act, w_mul, bias_mul, residual, out,
                    out_dtype, stream)


def grouped_linear(x, offsets, w, ws, bias=None, act="none", w_mul=None, bias_mul=None, residual=None, out=None,
                   out_dtype=None, stream=None):
    """linear of each group's rows with that group's weights: rows offsets[e] .. offsets[e+1] - 1
    take w[e]. offsets: int32 [E + 1] on the device (sort_pairs); w, w_mul: [E][N][K]; bias,
    bias_mul: [E][N]. Rows behind offsets[E] are neither used nor written (with out=None:
    uninitialised)."""
    E = w.shape[0]
    return _product(lib().dpa_grouped_linear, "dpa_grouped_linear", x, w, (E,), (E, offsets), ws, bias, act, w_mul,
                    bias_mul, residual, out, out_dtype, stream)


class DenseLayer:
    """One MoE layer at full precision (bf16 experts, nothing encoded) around the same router: the
    layer that the bitplane layer's budgets are compared with. Tensors on one device: w_gate, w_up
    [E][inter][hidden], w_down [E][hidden][inter], w_router [E][hidden], shared None or (gate, up
    [S][inter][hidden], down [S][hidden][inter]), all bf16 or int16 bits."""

    def __init__(self, desc: LayerDesc, w_gate, w_up, w_down, w_router, shared=None):
        if (0 if shared is None else len(shared[0])) != desc.n_shared:
            raise ValueError(f"shared: expected the weights of {desc.n_shared} always-on experts")
        self.desc = desc
        self.w_gate, self.w_up, self.w_down, self.w_router, self.shared = w_gate, w_up, w_down, w_router, shared

    @classmethod
    def from_host(cls, desc: LayerDesc, w_gate: np.ndarray, w_up: np.ndarray, w_down: np.ndarray,
                  w_router_bits: np.ndarray, shared_bits=None, device="cuda"):
        """From host fp32 experts (the arrays that encode takes), rounded to bf16 on the device, and
        bf16 bits of the router and the shared experts."""
        import torch

        def dev(a):
            return torch.from_numpy(np.ascontiguousarray(a)).to(device)

        gate, up, down = (dev(w.astype(np.float32, copy=False)).to(torch.bfloat16) for w in (w_gate, w_up, w_down))
        shared = None if shared_bits is None else tuple(dev(s.view(np.int16)).view(torch.bfloat16) for s in shared_bits)
        return cls(desc, gate, up, down, dev(w_router_bits.view(np.int16)), shared)

    def buffers(self, n_tokens: int):
        """Workspaces and intermediate rows of dense_moe_forward for n_tokens tokens."""
        import torch
        d, dev = self.desc, self.w_gate.device
        P = n_tokens * d.top_k

        def new(*shape, dtype):
            return torch.empty(shape, dtype=dtype, device=dev)

        bufs = {"ws": new_workspace(d, n_tokens, device=dev), "sort_ws": new_sort_workspace(P, d.n_experts, device=dev),
                "pos": new(n_tokens, d.top_k, dtype=torch.int32), "order": new(P, dtype=torch.int32),
                "offsets": new(d.n_experts + 1, dtype=torch.int32), "rows": new(P, d.hidden, dtype=torch.bfloat16),
                "h": new(P, d.inter, dtype=torch.bfloat16), "z": new(P, d.hidden, dtype=torch.float32)}
        if self.shared is not None:
            bufs["shared_h"] = new(n_tokens, d.inter, dtype=torch.bfloat16)
            bufs["shared_y"] = new(n_tokens, d.hidden, dtype=torch.float32)
        return bufs


def dense_moe_forward(layer: DenseLayer, x, bufs, y=None, aux: Optional[dict] = None, stream=None):
    """One MoE layer at full precision: route, sort the pairs by expert, the experts' gate/up with
    SwiGLU and down products on each expert's rows, and the gate-weighted sum back to the tokens, on
    top of the shared experts' outputs. x: CUDA int16/bf16 bits [T][H]; bufs: layer.buffers(T). aux:
    optional dict that receives "topk_idx" and "topk_gate". The SwiGLU output is rounded to bf16
    between the two products, every other intermediate is fp32. Returns y (int16 bf16 bits [T][H])."""
    import torch
    if stream is not None or x.get_device() != torch.cuda.current_device():
        dev = _device(x)
        if stream is not None and stream.device.index != dev:
            raise ValueError(f"stream: expected a stream of cuda:{dev}, got one of {stream.device}")
        # every buffer of the call, the router's outputs among them, belongs to the call's stream
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            return dense_moe_forward(layer, x, bufs, y, aux)
    # what the router reads is checked here, before the first launch
    desc, dev, ws = layer.desc, _device(x), bufs["ws"]
    _arg(x, "x", (len(x), desc.hidden), DTYPE_BF16, dev)
    _arg(layer.w_router, "w_router", (desc.n_experts, desc.hidden), DTYPE_BF16, dev)
    _workspace(ws, dev)
    if y is None:
        y = torch.empty(x.shape, dtype=torch.int16, device=x.device)
    else:
        _arg(y, "y", x.shape, DTYPE_BF16, dev)
    idx, gate = route(desc, x, layer.w_router, ws)
    if aux is not None:
        aux["topk_idx"], aux["topk_gate"] = idx, gate
    xb = x.view(torch.bfloat16)
    acc = None
    for s in range(desc.n_shared):
        g, u, d = (m[s] for m in layer.shared)
        linear(xb, g, ws, act="silu", w_mul=u, out=bufs["shared_h"])
        acc = linear(bufs["shared_h"], d, ws, residual=acc, out=bufs["shared_y"])
    sort_pairs(idx, desc.n_experts, bufs["sort_ws"], bufs["pos"], bufs["order"], bufs["offsets"])
    permute_rows(xb, bufs["pos"], out=bufs["rows"])
    grouped_linear(bufs["rows"], bufs["offsets"], layer.w_gate, ws, act="silu", w_mul=layer.w_up, out=bufs["h"])
    grouped_linear(bufs["h"], bufs["offsets"], layer.w_down, ws, out=bufs["z"])
    unpermute_rows(bufs["z"], bufs["pos"], gate, residual=acc, out=y)
    return y


def stream_prefixes(desc: LayerDesc, host_planes, host_meta, experts, kplanes, dev_planes, dev_meta,
                    stream=None) -> int:
    """Copy the first kplanes[i] planes (and their scale data) of experts[i] from the host
    layer (pinned torch uint8 tensors) to the device layer. Returns the bytes issued."""
    ex = np.ascontiguousarray(experts, dtype=np.int32)
    kp = np.ascontiguousarray(kplanes, dtype=np.uint8)
    nbytes = ctypes.c_uint64(0)
    _check(lib().dpa_stream_prefixes(ctypes.byref(desc), host_planes.data_ptr(), host_meta.data_ptr(), _ptr(ex),
                                     _ptr(kp), int(ex.size), _dptr(dev_planes), _dptr(dev_meta), ctypes.byref(nbytes),
                                     _stream(stream)), "dpa_stream_prefixes")
    return int(nbytes.value)


def solve_stored_widths(desc: LayerDesc, importance: np.ndarray, rtable: np.ndarray, budget_planes: int) -> np.ndarray:
    """Per-expert stored planes (uint8 [E]) minimising sum_e importance[e] * rtable[e][b_e - 1]
    within a budget of stored planes over all experts (host)."""
    imp = np.ascontiguousarray(importance, dtype=np.float64)
    r = np.ascontiguousarray(rtable, dtype=np.float64)
    w = np.zeros(desc.n_experts, dtype=np.uint8)
    _check(lib().dpa_solve_stored_widths(ctypes.byref(desc), _ptr(imp), _ptr(r), int(budget_planes), _ptr(w)),
           "dpa_solve_stored_widths")
    return w


def compact_layer(desc: LayerDesc, planes: np.ndarray, meta: np.ndarray, widths: np.ndarray):
    """Host compact layer for per-expert stored widths: (planes, meta, offsets uint64 [E][2])."""
    w = np.ascontiguousarray(widths, dtype=np.uint8)
    pb, mb = ctypes.c_uint64(0), ctypes.c_uint64(0)
    _check(lib().dpa_compact_sizes(ctypes.byref(desc), _ptr(w), ctypes.byref(pb), ctypes.byref(mb)),
           "dpa_compact_sizes")
    po = np.zeros(pb.value, dtype=np.uint8)
    mo = np.zeros(mb.value, dtype=np.uint8)
    off = np.zeros((desc.n_experts, 2), dtype=np.uint64)
    _check(lib().dpa_compact_layer(ctypes.byref(desc), _ptr(np.ascontiguousarray(planes)),
                                   _ptr(np.ascontiguousarray(meta)), _ptr(w), _ptr(po), _ptr(mo), _ptr(off)),
           "dpa_compact_layer")
    return po, mo, off


def device_error_detail(ws) -> Tuple[int, int]:
    """(code, detail) of the device error flag in ws, without clearing it (synchronises). The
    detail says which check or wait recorded it."""
    import torch
    torch.cuda.synchronize(ws.device)
    v = ws[:8].cpu().numpy().view(np.uint32)
    return int(v[0]), int(v[1])


def device_status(ws, stream=None) -> int:
    """Synchronise, read and clear the device error flag; returns the status code."""
    return int(lib().dpa_device_status(_dptr(ws), _stream(stream)))
