"""Python binding of libmoe_mi355x.so (C ABI in include/moe.h).

Argument marshalling only: every function passes torch tensors' device
pointers and torch's current HIP stream to the C entry point of the same name
and raises ``MoeError`` on a non-zero status. No step of the layer runs here.

torch is imported before the library is loaded so that the library binds to
the HIP runtime torch already loaded (one runtime per process: streams and
pointers are shared). The library must have been built
(``python -m token_choice_routing_amd.build``); importing the package does not
fall back to anything when it is missing.
"""
import ctypes
import importlib
import os
import re

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_mi355x.so")
MARSHAL_PATH = os.path.join(HERE, "_marshal.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "moe.h")

MOE_OK, MOE_ERR_ARG, MOE_ERR_ALIGN, MOE_ERR_WORKSPACE, MOE_ERR_UNSUPPORTED, MOE_ERR_HIP, MOE_ERR_NONFINITE = range(7)
MOE_F32, MOE_BF16, MOE_F16 = 0, 1, 2
MOE_NULL_ZERO, MOE_NULL_COPY, MOE_NULL_CONSTANT = 0, 1, 2
NULL_KINDS = {"zero": MOE_NULL_ZERO, "copy": MOE_NULL_COPY, "constant": MOE_NULL_CONSTANT}
(MOE_WS_LAYER, MOE_WS_ROUTE, MOE_WS_PERMUTE, MOE_WS_AUX, MOE_WS_BACKWARD,
 MOE_WS_COMBINE_BACKWARD, MOE_WS_STATE8, MOE_WS_TRAIN8) = range(8)
MOE_GEMM_GATE_UP, MOE_GEMM_DOWN = 0, 1


class MoeError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_str(status)})")


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d_model", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("n_null", ctypes.c_int32), ("top_k", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("d_ff_shared", ctypes.c_int32), ("dtype", ctypes.c_int32), ("null_kind", ctypes.c_int32)]


class LayerParams(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("w_router", ctypes.c_void_p), ("null_bias", ctypes.c_float),
                ("null_bias_tok", ctypes.c_void_p), ("w_gate", ctypes.c_void_p),
                ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p), ("ws_gate", ctypes.c_void_p),
                ("ws_up", ctypes.c_void_p), ("ws_down", ctypes.c_void_p), ("null_value", ctypes.c_void_p)]


class AuxOut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("logits", "topk_idx", "topk_w", "n_real", "offsets", "counts", "f", "P", "scalars")]


class LayerGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("dx", "dw_router", "dw_gate", "dw_up", "dw_down", "dws_gate", "dws_up", "dws_down")]


_lib = None
_marshal = None  # argument checks of the row operators (csrc/marshal.cpp), loaded on their first call
_P = ctypes.c_void_p


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run `python -m token_choice_routing_amd.build`")
    lib = ctypes.CDLL(path)
    D, I, L = ctypes.POINTER(Dims), ctypes.c_int32, ctypes.c_int64
    sig = {
        "moe_route": [D, _P, _P, ctypes.c_float, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_permute": [D, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_expert_ffn": [D, ctypes.c_int32, ctypes.c_int32, ctypes.c_int64, _P, _P, _P, _P, _P, _P,
                           _P, ctypes.c_size_t, _P],
        "moe_combine": [D, _P, _P, _P, _P, _P, _P, _P],
        "moe_expert_gate_up": [D, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P],
        "moe_grouped_gemm": [D, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                             ctypes.c_int64, _P, _P, _P, _P, _P, _P],
        "moe_combine_rows": [D, I, _P, _P, _P, _P, _P, _P, _P],
        "moe_combine_backward": [D, I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_permute_backward": [D, I, _P, _P, _P, I, _P, _P],
        "moe_act8_pack": [L, I, I, _P, L, _P, _P, _P, _P],
        "moe_act8_unpack": [L, I, I, _P, _P, _P, _P, L, _P],
        "moe_swiglu_keep8": [L, I, I, _P, _P, L, _P, _P, _P, _P, _P, _P, _P],
        "moe_swiglu_backward8": [L, I, _P, _P, _P, _P, _P, I, _P, _P, _P, L, I, _P, _P, L, _P, _P, _P],
        "moe_aux_stats": [D, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_layer_forward": [D, ctypes.POINTER(LayerParams), _P, ctypes.POINTER(AuxOut), _P,
                              ctypes.c_size_t, _P],
        "moe_layer_forward_noalloc": [D, ctypes.POINTER(LayerParams), _P, ctypes.POINTER(AuxOut), _P],
        "moe_layer_backward": [D, ctypes.POINTER(LayerParams), _P, ctypes.c_float, ctypes.c_float,
                               ctypes.POINTER(LayerGrads), _P, ctypes.c_size_t, _P],
        "moe_layer_forward_train": [D, ctypes.POINTER(LayerParams), _P, ctypes.POINTER(AuxOut), _P,
                                    ctypes.c_size_t, _P],
        "moe_layer_backward_saved": [D, ctypes.POINTER(LayerParams), _P, ctypes.c_float, ctypes.c_float,
                                     ctypes.POINTER(LayerGrads), _P, ctypes.c_size_t, _P],
        "moe_layer_forward_train8": [D, ctypes.POINTER(LayerParams), _P, ctypes.POINTER(AuxOut), _P,
                                     ctypes.c_size_t, _P, ctypes.c_size_t, _P],
        "moe_layer_backward_saved8": [D, ctypes.POINTER(LayerParams), _P, ctypes.c_float, ctypes.c_float,
                                      ctypes.POINTER(LayerGrads), _P, ctypes.c_size_t, _P, ctypes.c_size_t, _P],
        "moe_validate_inputs": [D, ctypes.POINTER(LayerParams), _P, ctypes.c_size_t, _P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.moe_workspace_bytes.argtypes = [D, ctypes.c_int32]
    lib.moe_workspace_bytes.restype = ctypes.c_size_t
    lib.moe_expert_ffn_workspace_bytes.argtypes = [D, ctypes.c_int32, ctypes.c_int64]
    lib.moe_expert_ffn_workspace_bytes.restype = ctypes.c_size_t
    lib.moe_status_str.argtypes = [ctypes.c_int]
    lib.moe_status_str.restype = ctypes.c_char_p
    lib.moe_version.argtypes = []
    lib.moe_version.restype = ctypes.c_int32
    _lib = lib
    return lib


def header_functions(path: str = HEADER):
    """Names of the functions include/moe.h declares."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_\w+)\s*\(", text)) - {"moe_stream"})


def _ptr(t):
    """Device address of a tensor argument (an int is taken as an address as is).
    The library reads every array as a dense row-major block in device memory, so a
    host tensor or a strided view is refused here rather than read wrongly there."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if t.device.type != "cuda":
        raise ValueError(f"expected a device tensor, got one on {t.device}")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor (the library reads dense row-major arrays)")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        if not torch.cuda.is_available():
            return None
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_ROW_TYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float16: MOE_F16}
_DTYPES = {v: k for k, v in _ROW_TYPES.items()}


# The calls below move rows and often take microseconds on the device, about as long as
# it takes to ask ten tensors from Python what they are: their arguments are checked in
# one native call, and what is wrong is worked out only when it refuses one. The library
# sees addresses only, so a tensor of another type or shape or on another device than the
# current one is refused here.

def _load_marshal():
    """The native checks. Only these calls need them: the layer's run without."""
    global _marshal
    if _marshal is None:
        build = "run `python -m token_choice_routing_amd.build`"
        if not os.path.exists(MARSHAL_PATH):
            raise ImportError(f"{MARSHAL_PATH} (argument checks of the row operators) is not built; {build}")
        try:
            _marshal = importlib.import_module("._marshal", __name__)
        except ImportError as e:
            raise ImportError(f"{MARSHAL_PATH} does not load with this torch, {build}: {e}") from e
    return _marshal


def _device():
    """Index of the current device; tensors of these calls have to be on it."""
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else 0


def _row_stream(stream, dev):
    """The stream of a call on device dev (torch's current one by default)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if isinstance(stream, int):
        return stream
    if getattr(stream, "device_index", dev) != dev:
        raise ValueError(f"stream: expected one of the current device (cuda:{dev}), got one of "
                         f"cuda:{stream.device_index}")
    return stream.cuda_stream


def _refuse(name, t, dev, dtype, shape, layout="a contiguous tensor"):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a tensor, got {type(t).__name__}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on the current device (cuda:{dev}), got one on {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: expected {layout}, got strides {t.stride()}")


def _dense(dev, names, *spec):
    """Device addresses of dense tensors; spec: a tensor (or None), its type and its shape
    for each name."""
    got = (_marshal or _load_marshal()).dense(dev, *spec)
    if got.__class__ is int:
        _refuse(names[got], spec[3 * got], dev, spec[3 * got + 1], spec[3 * got + 2])
    return got


def _matrix(name, t, dev, dtype, shape):
    """(device address, elements from row to row) of a [rows][cols] tensor whose rows may
    be spaced (a column range of a wider matrix) but are dense inside."""
    got = (_marshal or _load_marshal()).matrix(dev, t, dtype, shape)
    if got is None:
        _refuse(name, t, dev, dtype, shape, "rows that are dense and do not overlap")
    return got


def _matrix_like(name, t):
    """(type, shape) of a matrix that sets them for its call's other tensors."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype not in _ROW_TYPES:
        raise ValueError(f"{name}: expected a matrix of float32, bfloat16 or float16")
    return t.dtype, t.shape


def _row_dtype(name, code):
    if code not in _DTYPES:
        raise ValueError(f"{name}: expected MOE_F32, MOE_BF16 or MOE_F16, got {code}")
    return _DTYPES[code]


def _check(status, where):
    if status != MOE_OK:
        raise MoeError(status, where)


def _ws(ws):
    """(device address, bytes) of a workspace tensor, checked like every other
    tensor argument (device memory, contiguous); a tuple is taken as given."""
    if ws is None:
        return None, 0
    if isinstance(ws, tuple):
        return ws
    return _ptr(ws), ws.numel() * ws.element_size()


def status_str(status: int) -> str:
    return load_library().moe_status_str(int(status)).decode()


def version() -> int:
    return load_library().moe_version()


def make_dims(T, d_model, n_experts, n_null, top_k, d_ff, d_ff_shared=0, dtype=MOE_BF16,
              null_kind=MOE_NULL_ZERO) -> Dims:
    return Dims(int(T), int(d_model), int(n_experts), int(n_null), int(top_k), int(d_ff),
                int(d_ff_shared), int(dtype), int(null_kind))


def dims_from_config(cfg, T=None) -> Dims:
    return make_dims(cfg.T if T is None else T, cfg.d_model, cfg.n_experts, cfg.n_null, cfg.top_k,
                     cfg.d_ff, cfg.d_ff_shared, MOE_BF16 if cfg.dtype == "bf16" else MOE_F32,
                     NULL_KINDS[cfg.null_kind])


def workspace_bytes(dims: Dims, which: int = MOE_WS_LAYER) -> int:
    return load_library().moe_workspace_bytes(ctypes.byref(dims), which)


def expert_ffn_workspace_bytes(dims: Dims, d_ff: int, max_rows: int) -> int:
    return load_library().moe_expert_ffn_workspace_bytes(ctypes.byref(dims), d_ff, max_rows)


def moe_route(dims, x, w_router, null_bias=0.0, null_bias_tok=None, logits_in=None,
              logits_out=None, topk_idx=None, topk_w=None, n_real=None, ws=None, stream=None):
    wp, wb = _ws(ws)
    _check(load_library().moe_route(ctypes.byref(dims), _ptr(x), _ptr(w_router), float(null_bias),
                                     _ptr(null_bias_tok), _ptr(logits_in), _ptr(logits_out),
                                     _ptr(topk_idx), _ptr(topk_w), _ptr(n_real), wp, wb,
                                     _stream(stream)), "moe_route")


def moe_permute(dims, topk_idx, x, counts, offsets, perm_token, slot_pos, x_perm, ws, stream=None):
    wp, wb = _ws(ws)
    _check(load_library().moe_permute(ctypes.byref(dims), _ptr(topk_idx), _ptr(x), _ptr(counts),
                                       _ptr(offsets), _ptr(perm_token), _ptr(slot_pos),
                                       _ptr(x_perm), wp, wb, _stream(stream)), "moe_permute")


def moe_expert_ffn(dims, n_groups, d_ff, max_rows, a, offsets, w_gate, w_up, w_down, out, ws,
                   stream=None):
    wp, wb = _ws(ws)
    _check(load_library().moe_expert_ffn(ctypes.byref(dims), int(n_groups), int(d_ff), int(max_rows),
                                          _ptr(a), _ptr(offsets), _ptr(w_gate), _ptr(w_up),
                                          _ptr(w_down), _ptr(out), wp, wb, _stream(stream)),
           "moe_expert_ffn")


def moe_grouped_gemm(dims, op, n_groups, n_out, k_dim, rows, a, offsets, b0, b1, out, stream=None):
    _check(load_library().moe_grouped_gemm(ctypes.byref(dims), int(op), int(n_groups), int(n_out),
                                            int(k_dim), int(rows), _ptr(a), _ptr(offsets), _ptr(b0),
                                            _ptr(b1), _ptr(out), _stream(stream)), "moe_grouped_gemm")


def moe_expert_gate_up(dims, x, perm_token, offsets, w_gate, w_up, ws_gate, ws_up, h, hs, stream=None):
    _check(load_library().moe_expert_gate_up(ctypes.byref(dims), _ptr(x), _ptr(perm_token), _ptr(offsets),
                                              _ptr(w_gate), _ptr(w_up), _ptr(ws_gate), _ptr(ws_up), _ptr(h),
                                              _ptr(hs), _stream(stream)), "moe_expert_gate_up")


def moe_combine(dims, y_perm, slot_pos, topk_w, y_shared, y, stream=None, null_src=None):
    """null_src: the rows a null slot adds (x for copy experts, v for constant)."""
    _check(load_library().moe_combine(ctypes.byref(dims), _ptr(y_perm), _ptr(slot_pos),
                                       _ptr(topk_w), _ptr(y_shared), _ptr(null_src), _ptr(y),
                                       _stream(stream)),
           "moe_combine")


def _slot_shapes(dims):
    """(dims dtype, [T][d], slots [T][K], rows in expert order, null source) of a dispatch call."""
    T, K, d, N = dims.T, dims.top_k, dims.d_model, dims.n_experts
    return (_DTYPES.get(dims.dtype), (T, d), (T, K), (T * (K if K < N else N), d),
            (d,) if dims.null_kind == MOE_NULL_CONSTANT else (T, d))


_COMBINE_ROWS = ("y_perm", "slot_pos", "topk_w", "y_shared", "null_src", "y")


def moe_combine_rows(dims, rows_dtype, y_perm, slot_pos, topk_w, y_shared, y, null_src=None, stream=None):
    """moe_combine with y_perm and y_shared of type rows_dtype (MOE_F32, MOE_BF16 or
    MOE_F16). null_src: the rows a null slot adds (x for copy experts, v for constant)."""
    lib, dev = load_library(), _device()
    dt, token, slots, rows, nul = _slot_shapes(dims)
    rt = _row_dtype("rows_dtype", rows_dtype)
    ptrs = _dense(dev, _COMBINE_ROWS, y_perm, rt, rows, slot_pos, torch.int32, slots, topk_w, torch.float32, slots,
                  y_shared, rt, token, null_src if dims.null_kind else None, dt, nul, y, dt, token)
    _check(lib.moe_combine_rows(ctypes.byref(dims), rows_dtype, *ptrs, _row_stream(stream, dev)), "moe_combine_rows")


_COMBINE_BACKWARD = ("dy", "y_perm", "slot_pos", "topk_w", "null_src", "dy_perm", "w_perm", "row_slot", "dtopk_w",
                     "dnull")


def moe_combine_backward(dims, rows_dtype, dy, y_perm, slot_pos, topk_w, dy_perm=None, w_perm=None, row_slot=None,
                         dtopk_w=None, null_src=None, dnull=None, ws=None, stream=None):
    """Gradients of moe_combine / moe_combine_rows: dy_perm (rows_dtype), dtopk_w and the
    null source's dnull; w_perm and row_slot hold each expert row's weight and flat slot
    index. Every output is optional. ws: MOE_WS_COMBINE_BACKWARD bytes (constant nulls
    with dnull)."""
    lib, dev, f32, i32 = load_library(), _device(), torch.float32, torch.int32
    dt, token, slots, rows, nul = _slot_shapes(dims)
    rt = _row_dtype("rows_dtype", rows_dtype)
    if not dims.null_kind:
        null_src = dnull = None
    ptrs = _dense(dev, _COMBINE_BACKWARD, dy, dt, token, y_perm, rt, rows, slot_pos, i32, slots, topk_w, f32, slots,
                  null_src, dt, nul, dy_perm, rt, rows, w_perm, f32, rows[:1], row_slot, i32, rows[:1],
                  dtopk_w, f32, slots, dnull, f32, nul)
    wp, wb = _ws(ws)
    _check(lib.moe_combine_backward(ctypes.byref(dims), rows_dtype, *ptrs, wp, wb, _row_stream(stream, dev)),
           "moe_combine_backward")


_PERMUTE_BACKWARD = ("dx_perm", "slot_pos", "dx_add", "dx")


def moe_permute_backward(dims, rows_dtype, dx_perm, slot_pos, dx_add, dx_dtype, dx, stream=None):
    """Gradient of moe_permute's gather: dx = dx_add (float32, optional) + the sum of each
    token's real rows of dx_perm (rows_dtype), in dx_dtype; dx may be dx_add itself."""
    lib, dev = load_library(), _device()
    _, token, slots, rows, _ = _slot_shapes(dims)
    rt, dt = _row_dtype("rows_dtype", rows_dtype), _row_dtype("dx_dtype", dx_dtype)
    pp, ps, pa, px = _dense(dev, _PERMUTE_BACKWARD, dx_perm, rt, rows, slot_pos, torch.int32, slots,
                            dx_add, torch.float32, token, dx, dt, token)
    _check(lib.moe_permute_backward(ctypes.byref(dims), rows_dtype, pp, ps, pa, dx_dtype, px,
                                    _row_stream(stream, dev)), "moe_permute_backward")


ACT8_BLOCK = 32  # columns that share a scale byte
_COUNT = (1,)


def act8_scales_shape(rows, cols):
    """Shape of the uint8 scales of a [rows][cols] checkpoint (its codes are int8 [rows][cols])."""
    return rows, -(-cols // ACT8_BLOCK)


_ACT8 = ("n_rows", "codes", "scales")


def moe_act8_pack(x, codes, scales, n_rows=None, stream=None):
    """8-bit checkpoint of x [rows][cols] (float32, bfloat16 or float16; rows may be
    spaced): codes int8 [rows][cols], scales uint8 [rows][ceil(cols / 32)]. n_rows: device
    int32 [1], the rows in use (all if None); the others are left as they were."""
    lib, dev = load_library(), _device()
    dt, shape = _matrix_like("x", x)
    rows, cols = shape
    px, ld = _matrix("x", x, dev, dt, shape)
    pn, pc, ps = _dense(dev, _ACT8, n_rows, torch.int32, _COUNT, codes, torch.int8, shape,
                        scales, torch.uint8, act8_scales_shape(rows, cols))
    _check(lib.moe_act8_pack(rows, cols, _ROW_TYPES[dt], px, ld, pn, pc, ps, _row_stream(stream, dev)),
           "moe_act8_pack")


def moe_act8_unpack(codes, scales, out, n_rows=None, stream=None):
    """The values a checkpoint stands for, into out [rows][cols] (rows may be spaced)."""
    lib, dev = load_library(), _device()
    dt, shape = _matrix_like("out", out)
    rows, cols = shape
    po, ld = _matrix("out", out, dev, dt, shape)
    pn, pc, ps = _dense(dev, _ACT8, n_rows, torch.int32, _COUNT, codes, torch.int8, shape,
                        scales, torch.uint8, act8_scales_shape(rows, cols))
    _check(lib.moe_act8_unpack(rows, cols, _ROW_TYPES[dt], pc, ps, pn, po, ld, _row_stream(stream, dev)),
           "moe_act8_unpack")


_KEEP8 = ("n_rows", "h", "g_codes", "g_scales", "u_codes", "u_scales")


def moe_swiglu_keep8(g, u, h, g_codes, g_scales, u_codes, u_scales, n_rows=None, stream=None):
    """h = silu(g) u and the 8-bit checkpoints of g and u. g, u: [rows][d_ff] of one type,
    with the same spacing of rows; h: dense, the same type."""
    lib, dev, i8, u8 = load_library(), _device(), torch.int8, torch.uint8
    dt, shape = _matrix_like("g", g)
    rows, F = shape
    pg, ld = _matrix("g", g, dev, dt, shape)
    pu, ldu = _matrix("u", u, dev, dt, shape)
    if ld != ldu:
        raise ValueError(f"g and u: expected the same spacing of rows, got {ld} and {ldu}")
    scaled = act8_scales_shape(rows, F)
    ptrs = _dense(dev, _KEEP8, n_rows, torch.int32, _COUNT, h, dt, shape, g_codes, i8, shape, g_scales, u8, scaled,
                  u_codes, i8, shape, u_scales, u8, scaled)
    _check(lib.moe_swiglu_keep8(rows, F, _ROW_TYPES[dt], pg, pu, ld, *ptrs, _row_stream(stream, dev)),
           "moe_swiglu_keep8")


_BACKWARD8 = ("g_codes", "g_scales", "u_codes", "u_scales", "n_rows", "dh", "w_rows", "row_slot", "h", "dw")


def moe_swiglu_backward8(g_codes, g_scales, u_codes, u_scales, dh, dg, du, h=None, w_rows=None, dw=None,
                         row_slot=None, n_rows=None, stream=None):
    """The SwiGLU backward from the checkpoints of g and u: dg, du (one type, rows may be
    spaced alike), optionally h (the same type, dense) and dw = <dh, h> per row (at
    dw[row_slot[p]] when row_slot is given). w_rows scales dh per row in dg and du."""
    lib, dev, f32, i32, i8, u8 = load_library(), _device(), torch.float32, torch.int32, torch.int8, torch.uint8
    dt, shape = _matrix_like("dg", dg)
    rows, F = shape
    pg, ld = _matrix("dg", dg, dev, dt, shape)
    pu, ldu = _matrix("du", du, dev, dt, shape)
    if ld != ldu:
        raise ValueError(f"dg and du: expected the same spacing of rows, got {ld} and {ldu}")
    tdh, _ = _matrix_like("dh", dh)
    n_slots, dw_shape = 0, None
    if dw is not None:
        n_slots, dw_shape = dw.numel(), dw.shape
        if row_slot is None and n_slots != rows:
            raise ValueError(f"dw: expected {rows} elements, got {n_slots}")
    scaled, col = act8_scales_shape(rows, F), (rows,)
    cg, sg, cu, su, pn, pd, pw, pr, ph, pdw = _dense(
        dev, _BACKWARD8, g_codes, i8, shape, g_scales, u8, scaled, u_codes, i8, shape, u_scales, u8, scaled,
        n_rows, i32, _COUNT, dh, tdh, shape, w_rows, f32, col, row_slot, i32, col, h, dt, shape, dw, f32, dw_shape)
    _check(lib.moe_swiglu_backward8(rows, F, cg, sg, cu, su, pn, _ROW_TYPES[tdh], pd, pw, pr, n_slots, _ROW_TYPES[dt],
                                    pg, pu, ld, ph, pdw, _row_stream(stream, dev)), "moe_swiglu_backward8")


def moe_aux_stats(dims, logits, topk_idx, f, P, counts, scalars, ws, stream=None):
    wp, wb = _ws(ws)
    _check(load_library().moe_aux_stats(ctypes.byref(dims), _ptr(logits), _ptr(topk_idx), _ptr(f),
                                         _ptr(P), _ptr(counts), _ptr(scalars), wp, wb,
                                         _stream(stream)), "moe_aux_stats")


def moe_layer_forward(dims, params: LayerParams, y, aux: AuxOut = None, ws=None, stream=None):
    wp, wb = _ws(ws)
    _check(load_library().moe_layer_forward(ctypes.byref(dims), ctypes.byref(params), _ptr(y),
                                             ctypes.byref(aux) if aux is not None else None, wp, wb,
                                             _stream(stream)), "moe_layer_forward")


MOE_NOALLOC_MAX_WS_BYTES = 64 << 20


def moe_layer_forward_noalloc(dims, params: LayerParams, y, aux: AuxOut = None, stream=None):
    """moe_layer_forward with the library's static per-device workspace (no allocation)."""
    _check(load_library().moe_layer_forward_noalloc(ctypes.byref(dims), ctypes.byref(params), _ptr(y),
                                                     ctypes.byref(aux) if aux is not None else None,
                                                     _stream(stream)), "moe_layer_forward_noalloc")


def moe_layer_backward(dims, params: LayerParams, dy, alpha: float, beta: float, grads: LayerGrads,
                       ws=None, stream=None):
    wp, wb = _ws(ws)
    _check(load_library().moe_layer_backward(ctypes.byref(dims), ctypes.byref(params), _ptr(dy),
                                              float(alpha), float(beta), ctypes.byref(grads), wp, wb,
                                              _stream(stream)), "moe_layer_backward")


def moe_layer_forward_train(dims, params: LayerParams, y, aux: AuxOut = None, ws=None, stream=None):
    """The layer forward that leaves its routing and expert pre-activations in ws (the
    backward's workspace) for moe_layer_backward_saved."""
    wp, wb = _ws(ws)
    _check(load_library().moe_layer_forward_train(ctypes.byref(dims), ctypes.byref(params), _ptr(y),
                                                   ctypes.byref(aux) if aux is not None else None, wp, wb,
                                                   _stream(stream)), "moe_layer_forward_train")


def moe_layer_backward_saved(dims, params: LayerParams, dy, alpha: float, beta: float, grads: LayerGrads,
                             ws=None, stream=None):
    """moe_layer_backward from the state a moe_layer_forward_train call left in ws."""
    wp, wb = _ws(ws)
    _check(load_library().moe_layer_backward_saved(ctypes.byref(dims), ctypes.byref(params), _ptr(dy),
                                                    float(alpha), float(beta), ctypes.byref(grads), wp, wb,
                                                    _stream(stream)), "moe_layer_backward_saved")


def moe_layer_forward_train8(dims, params: LayerParams, y, aux: AuxOut = None, state=None, ws=None, stream=None):
    """The training forward that keeps its state in 8 bits in state (MOE_WS_STATE8 bytes)
    for moe_layer_backward_saved8; ws (MOE_WS_TRAIN8 bytes) is scratch of the call."""
    (sp, sb), (wp, wb) = _ws(state), _ws(ws)
    _check(load_library().moe_layer_forward_train8(ctypes.byref(dims), ctypes.byref(params), _ptr(y),
                                                    ctypes.byref(aux) if aux is not None else None, sp, sb, wp, wb,
                                                    _stream(stream)), "moe_layer_forward_train8")


def moe_layer_backward_saved8(dims, params: LayerParams, dy, alpha: float, beta: float, grads: LayerGrads,
                              state=None, ws=None, stream=None):
    """moe_layer_backward from the 8-bit state a moe_layer_forward_train8 call left in state."""
    (sp, sb), (wp, wb) = _ws(state), _ws(ws)
    _check(load_library().moe_layer_backward_saved8(ctypes.byref(dims), ctypes.byref(params), _ptr(dy),
                                                     float(alpha), float(beta), ctypes.byref(grads), sp, sb, wp, wb,
                                                     _stream(stream)), "moe_layer_backward_saved8")


def moe_validate_inputs(dims, params: LayerParams, ws, stream=None) -> bool:
    """True when the layer's inputs hold no NaN or infinity (null biases may be
    infinite), False when they do; synchronises the stream. ws: >= 16 device bytes."""
    wp, wb = _ws(ws)
    status = load_library().moe_validate_inputs(ctypes.byref(dims), ctypes.byref(params), wp, wb,
                                                _stream(stream))
    if status == MOE_ERR_NONFINITE:
        return False
    _check(status, "moe_validate_inputs")
    return True


from .layer import MoeLayer  # noqa: E402,F401
