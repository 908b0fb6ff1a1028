"""Python binding of libmoe: one GPU's MoE feed-forward layer on MI355X (gfx950).

Thin ctypes marshalling over the C ABI in ``include/moe.h``: every function
below has the name of the C entry point it calls, takes torch tensors that
already live on the GPU, passes their data pointers, sizes and the current
HIP stream, and raises ``MoeError`` on a non-OK status.  No computation
happens here and there is no CPU fallback: if ``libmoe.so`` has not been
built, importing the functions that need it raises ``ImportError``.

Build the library in-tree with ``python -m routing_grouped_gemm_amd.build``.
"""
import ctypes
import os

import torch

MOE_OK, MOE_EINVAL, MOE_EALIGN, MOE_EUNSUPPORTED, MOE_EWORKSPACE, MOE_EHIP = 0, -1, -2, -3, -4, -5
MOE_F32, MOE_BF16, MOE_MXFP8, MOE_MXFP4 = 0, 1, 2, 3
MOE_INT4 = 4   # of MoELayer (moe_int4_ffn has no dtype argument)
MOE_ERR_NONFINITE_LOGIT, MOE_ERR_ROW_RANGE = 1, 2

MOE_ACT_SILU, MOE_ACT_GELU, MOE_ACT_GELU_TANH, MOE_ACT_RELU = 0, 1, 2, 3

MOE_GEMM_GATE_UP, MOE_GEMM_DOWN, MOE_GEMM_DGRAD_DOWN, MOE_GEMM_DGRAD_GATE_UP, MOE_GEMM_WGRAD = \
    0, 1, 2, 3, 4

ABI_FUNCTIONS = ("moe_route_workspace_bytes", "moe_route_topk", "moe_route_topk_noalloc", "moe_permute",
                 "moe_gemm_workspace_bytes", "moe_grouped_gemm_fwd", "moe_grouped_gemm_bwd",
                 "moe_grouped_gemm_op", "moe_unpermute_combine", "moe_quantize_mxfp8",
                 "moe_quantize_mxfp4", "moe_dequantize_mxfp4", "moe_route_add_shared", "moe_router_logits",
                 "moe_gate_grad", "moe_dropout", "moe_combine_dropout", "moe_grouped_glu_op", "moe_grouped_glu_fwd",
                 "moe_grouped_glu_bwd", "moe_quantize_int4", "moe_dequantize_int4", "moe_int4_workspace_bytes",
                 "moe_int4_ffn", "moe_balance_workspace_bytes", "moe_balance_loss", "moe_balance_loss_bwd",
                 "moe_status_string", "moe_version")

GEMM_TENSOR_FIELDS = ("x_perm", "x_perm_scales", "w13", "w13_scales", "w2", "w2_scales", "gu",
                      "h", "y_perm", "dy_perm", "dgu", "dx_perm", "dw13", "dw2", "ws")
GEMM_TENSOR_FIELDS_F32 = ("dw13_f32", "dw2_f32")   # after ws_bytes: fp32 weight-gradient accumulators


class MoeGemmTensors(ctypes.Structure):
    """C struct moe_gemm_tensors (device pointers, NULL where unused); made by gemm_tensors(), which keeps
    the tensors with it, so that the calls can check them."""
    _fields_ = [(n, ctypes.c_void_p) for n in GEMM_TENSOR_FIELDS] + [("ws_bytes", ctypes.c_size_t)] + \
        [(n, ctypes.c_void_p) for n in GEMM_TENSOR_FIELDS_F32]
    given = checked = dev = None   # the tensors by name; the sizes they were last checked for, and their GPU


class MoeGlu(ctypes.Structure):
    """C struct moe_glu; made by glu(), which keeps the rng tensor alive with it."""
    _fields_ = [("act", ctypes.c_int), ("limit", ctypes.c_float), ("p", ctypes.c_float), ("rng", ctypes.c_void_p)]
    rng_tensor = None


class MoeInt4(ctypes.Structure):
    """C struct moe_int4."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p)]


_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")
_lib = None


class MoeError(RuntimeError):
    def __init__(self, status, name):
        self.status = status
        msg = load().moe_status_string(status).decode()
        super().__init__(f"{name} returned {status}: {msg}")


def load():
    """Load libmoe.so (once).  Raises ImportError if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m routing_grouped_gemm_amd.build` (there is no fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    lib.moe_version.restype = I
    lib.moe_version.argtypes = []
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_status_string.argtypes = [I]
    lib.moe_route_workspace_bytes.restype = SZ
    lib.moe_route_workspace_bytes.argtypes = [I, I, I]
    lib.moe_route_topk.restype = I
    lib.moe_route_topk.argtypes = [P, I, I, I, I, P, P, P, P, P, P, I64, P, SZ, P, P]
    lib.moe_route_topk_noalloc.restype = I
    lib.moe_route_topk_noalloc.argtypes = [P, I, I, I, I, P, P, P, P, P, P, I64, P, P]
    lib.moe_permute.restype = I
    lib.moe_permute.argtypes = [I, P, I, I, I, P, P, P, I64, P, P, P, P]
    lib.moe_gemm_workspace_bytes.restype = SZ
    lib.moe_gemm_workspace_bytes.argtypes = [I, I, I64, I, I]
    lib.moe_grouped_gemm_fwd.restype = I
    lib.moe_grouped_gemm_fwd.argtypes = [I, P, P, P, P, P, P, P, I, I, I64, I, I, P, P, P, P, SZ, P]
    lib.moe_grouped_gemm_bwd.restype = I
    lib.moe_grouped_gemm_bwd.argtypes = [I, P, P, P, P, P, P, P, P, P, P, I, I, I64, I, I, P, P, P,
                                         P, P, SZ, P]
    lib.moe_grouped_gemm_op.restype = I
    lib.moe_grouped_gemm_op.argtypes = [I, I, ctypes.POINTER(MoeGemmTensors), P, I, I, I64, I, I,
                                        P]
    lib.moe_unpermute_combine.restype = I
    lib.moe_unpermute_combine.argtypes = [I, P, P, P, I, I, I, I64, P, P, P]
    lib.moe_quantize_mxfp8.restype = I
    lib.moe_quantize_mxfp8.argtypes = [P, I64, I, I, P, I, P, P, P]
    lib.moe_route_add_shared.restype = I
    lib.moe_route_add_shared.argtypes = [I, I, I, I, I, P, P, P, P, P, P, I64, P, P, P, P, P, P, P]
    lib.moe_router_logits.restype = I
    lib.moe_router_logits.argtypes = [P, P, I, I, I, P, P]
    lib.moe_gate_grad.restype = I
    lib.moe_gate_grad.argtypes = [P, P, P, P, P, I, I, I, I, I64, P, P, P, P, P]
    F = ctypes.c_float
    lib.moe_dropout.restype = I
    lib.moe_dropout.argtypes = [I, P, P, I64, F, P, P, P]
    lib.moe_combine_dropout.restype = I
    lib.moe_combine_dropout.argtypes = [I, P, P, P, P, I, I, I, I64, F, P, P, P, P]
    GP = ctypes.POINTER(MoeGlu)
    lib.moe_grouped_glu_op.restype = I
    lib.moe_grouped_glu_op.argtypes = [I, I, GP, ctypes.POINTER(MoeGemmTensors), P, I, I, I64, I, I, P]
    lib.moe_grouped_glu_fwd.restype = I
    lib.moe_grouped_glu_fwd.argtypes = [I, GP, P, P, P, P, I, I, I64, I, I, P, P, P, P]
    lib.moe_grouped_glu_bwd.restype = I
    lib.moe_grouped_glu_bwd.argtypes = [I, GP, P, P, P, P, P, P, P, I, I, I64, I, I, P, P, P, P, P, SZ, P]
    lib.moe_quantize_int4.restype = I
    lib.moe_quantize_int4.argtypes = [P, I64, I, I, P, P, P, P]
    lib.moe_dequantize_int4.restype = I
    lib.moe_dequantize_int4.argtypes = [P, P, P, I64, I, I, P, P]
    lib.moe_int4_workspace_bytes.restype = SZ
    lib.moe_int4_workspace_bytes.argtypes = [I64, I, I]
    lib.moe_int4_ffn.restype = I
    lib.moe_int4_ffn.argtypes = [GP, P, I, I, P, P, P, P, P, I, I, I, I, ctypes.POINTER(MoeInt4),
                                 ctypes.POINTER(MoeInt4), P, P, SZ, P, P]
    lib.moe_quantize_mxfp4.restype = I
    lib.moe_quantize_mxfp4.argtypes = [P, I64, I, P, P, P]
    lib.moe_dequantize_mxfp4.restype = I
    lib.moe_dequantize_mxfp4.argtypes = [P, P, I64, I, P, P]
    lib.moe_balance_workspace_bytes.restype = SZ
    lib.moe_balance_workspace_bytes.argtypes = [I, I, I]
    lib.moe_balance_loss.restype = I
    lib.moe_balance_loss.argtypes = [P, P, P, P, I, I, I, I, F, F, P, P, P, P, P, P, SZ, P, P]
    lib.moe_balance_loss_bwd.restype = I
    lib.moe_balance_loss_bwd.argtypes = [P, P, P, I, I, I, P, P, F, F, P, P, P, P]
    _lib = lib
    return lib


def lib_path():
    return LIB_PATH


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# the current stream's handle without building a torch.cuda.Stream object: 0.4 us a call instead of 2.8
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _s(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(rc, name):
    if rc != MOE_OK:
        raise MoeError(rc, name)


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _dense(name, t, dtype, *shape):
    """The data pointer of t (None: NULL) after checking that it is a dense `dtype` tensor
    of `shape`."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {shape}, got {t.dtype} "
                         f"{tuple(t.shape)} with strides {t.stride()}")
    return t.data_ptr()


def _array(name, t, dtype, n):
    """The data pointer of t (None: NULL; a device pointer passes) after checking that it is a dense `dtype`
    tensor, of whatever shape, of the n elements at least that a kernel reads or writes there."""
    if t is None or isinstance(t, int):
        return t
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of {n} elements, got {t.dtype} "
                         f"{tuple(t.shape)} with strides {t.stride()}")
    return t.data_ptr()


def _byte_array(name, t, n):
    """_array of n bytes in any one-byte type (8-bit codes and scales)."""
    if t is None or isinstance(t, int):
        return t
    if t.element_size() != 1 or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor of {n} bytes, got {t.dtype} {tuple(t.shape)} with "
                         f"strides {t.stride()}")
    return t.data_ptr()


_I32 = torch.int32


def _call(name, stream, tensors, *args):
    """The C entry point `name` on `stream` (None: the current one of the tensors' device), with that
    device current; `tensors` must be on one GPU.  The stream is the last argument."""
    dev = tensors[0].get_device()
    if dev < 0:
        raise ValueError(f"{name}: expected tensors on a GPU, got one on {tensors[0].device}")
    for t in tensors:
        if t is not None and not isinstance(t, int) and t.get_device() != dev:
            raise ValueError(f"{name}: tensors on {tensors[0].device} and {t.device}")
    _launch(name, dev, stream, args)


def _launch(name, dev, stream, args):
    """The C entry point `name` on `stream` (None: the current one of the GPU dev), with dev current."""
    fn = getattr(load(), name)
    if dev == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(dev) if stream is None and _raw_stream else _s(stream))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _s(stream))
    if rc != MOE_OK:
        raise MoeError(rc, name)


# ------------------------------------------------------------------ ABI calls
def moe_version():
    return load().moe_version()


def moe_status_string(status):
    return load().moe_status_string(status).decode()


def moe_route_workspace_bytes(T, E, k):
    return int(load().moe_route_workspace_bytes(T, E, k))


def _route_args(logits, k, capacity, topk_idx, topk_w, counts, offsets, dst_row, src_slot):
    T, E = logits.shape
    return (_array("logits", logits, torch.float32, T * E), T, E, k, capacity, _array("topk_idx", topk_idx, _I32, T * k),
            _array("topk_w", topk_w, torch.float32, T * k), _array("counts", counts, _I32, E),
            _array("offsets", offsets, _I32, E + 1), _array("dst_row", dst_row, _I32, T * k),
            _array("src_slot", src_slot, _I32, 0), src_slot.numel())


def moe_route_topk(logits, k, capacity, topk_idx, topk_w, counts, offsets, dst_row, src_slot, ws,
                   dev_err=None, stream=None):
    """logits [T, E] fp32 -> topk_idx [T,k] i32, topk_w [T,k] f32, counts [E], offsets [E+1],
    dst_row [T*k], src_slot [n_rows] (n_rows = T*k, or E*capacity when padded)."""
    _call("moe_route_topk", stream, (logits, topk_idx, topk_w, counts, offsets, dst_row, src_slot, ws, dev_err),
          *_route_args(logits, k, capacity, topk_idx, topk_w, counts, offsets, dst_row, src_slot), _p(ws), _nbytes(ws),
          _array("dev_err", dev_err, _I32, 1))


ROUTE_NOALLOC_MAX_BYTES = 32 << 20    # MOE_ROUTE_NOALLOC_MAX_BYTES in moe.h


def moe_route_topk_noalloc(logits, k, capacity, topk_idx, topk_w, counts, offsets, dst_row, src_slot,
                           dev_err=None, stream=None):
    """moe_route_topk with the library's fixed per-GPU scratch instead of a workspace."""
    _call("moe_route_topk_noalloc", stream, (logits, topk_idx, topk_w, counts, offsets, dst_row, src_slot, dev_err),
          *_route_args(logits, k, capacity, topk_idx, topk_w, counts, offsets, dst_row, src_slot),
          _array("dev_err", dev_err, _I32, 1))


def moe_permute(dtype, x, k, dst_row, x_perm, src_slot=None, row_scale=None, x_perm_scales=None,
                dev_err=None, stream=None):
    """x [T, d] -> x_perm [n_rows, d] (MXFP8: codes + x_perm_scales [n_rows, d/32]; MXFP4:
    codes [n_rows, d/2] + x_perm_scales [n_rows, d/32]).  src_slot [n_rows]: for a padded
    layout; rows with src_slot < 0 become zero."""
    T, d = x.shape
    n_rows = x_perm.shape[0]
    if dtype == MOE_MXFP4:
        if dst_row.numel() != T * k:
            raise ValueError(f"dst_row: expected {T * k} rows for {T} tokens, got {dst_row.numel()}")
        _call("moe_permute", stream, (x, dst_row, x_perm, src_slot, row_scale, x_perm_scales, dev_err), dtype,
              _dense("x", x, torch.bfloat16, T, d), T, d, k, _dense("dst_row", dst_row, torch.int32, *dst_row.shape),
              _dense("src_slot", src_slot, torch.int32, n_rows), _p(row_scale), n_rows,
              _dense("x_perm", x_perm, torch.uint8, n_rows, d // 2),
              _dense("x_perm_scales", x_perm_scales, torch.uint8, n_rows, d // 32), _p(dev_err))
        return
    if torch.is_tensor(src_slot) and src_slot.numel() != n_rows:
        raise ValueError(f"src_slot: expected {n_rows} rows, as x_perm has, got {src_slot.numel()}")
    if dtype == MOE_MXFP8:
        t, out, scales = torch.bfloat16, _byte_array("x_perm", x_perm, n_rows * d), \
            _byte_array("x_perm_scales", x_perm_scales, n_rows * (d // 32))
    else:
        t = _float_type(dtype)
        out, scales = _array("x_perm", x_perm, t, n_rows * d), _p(x_perm_scales)
    _call("moe_permute", stream, (x, dst_row, x_perm, src_slot, row_scale, x_perm_scales, dev_err), dtype,
          _array("x", x, t, T * d), T, d, k, _array("dst_row", dst_row, _I32, T * k),
          _array("src_slot", src_slot, _I32, n_rows), _array("row_scale", row_scale, torch.float32, T * k), n_rows, out,
          scales, _array("dev_err", dev_err, _I32, 1))


def moe_gemm_workspace_bytes(dtype, E, n_rows, d, f):
    return int(load().moe_gemm_workspace_bytes(dtype, E, n_rows, d, f))


def _gemm_types(dtype):
    """Type of a grouped GEMM's activations, and the check of what it multiplies (MXFP8: codes)."""
    if dtype == MOE_MXFP8:
        return torch.bfloat16, _byte_array
    t = _float_type(dtype)
    return t, lambda name, w, n: _array(name, w, t, n)


def moe_grouped_gemm_fwd(dtype, x_perm, w13, w2, group_off, capacity, gu, h, y_perm,
                         x_perm_scales=None, w13_scales=None, w2_scales=None, ws=None,
                         stream=None):
    """x_perm [n_rows, d], w13 [E, 2f, d], w2 [E, d, f] -> gu [n_rows, 2f], h [n_rows, f],
    y_perm [n_rows, d].  group_off [E+1] device int32 (ignored when capacity > 0, but its
    length still gives E).  MXFP4: x_perm, w13 and w2 are codes, two elements per byte, and
    gu and h may be None (then not written)."""
    E = group_off.numel() - 1
    n_rows, d = x_perm.shape
    if dtype == MOE_MXFP4:
        d, f = 2 * d, 2 * w2.shape[-1]
        u8, bf = torch.uint8, torch.bfloat16
        _call("moe_grouped_gemm_fwd", stream, (x_perm, x_perm_scales, w13, w13_scales, w2, w2_scales, group_off, gu, h,
                                               y_perm, ws), dtype, _dense("x_perm", x_perm, u8, n_rows, d // 2),
              _dense("x_perm_scales", x_perm_scales, u8, n_rows, d // 32), _dense("w13", w13, u8, E, 2 * f, d // 2),
              _dense("w13_scales", w13_scales, u8, E, 2 * f, d // 32), _dense("w2", w2, u8, E, d, f // 2),
              _dense("w2_scales", w2_scales, u8, E, d, f // 32), _dense("group_off", group_off, torch.int32, E + 1),
              capacity, E, n_rows, d, f, _dense("gu", gu, bf, n_rows, 2 * f), _dense("h", h, bf, n_rows, f),
              _dense("y_perm", y_perm, bf, n_rows, d), _p(ws), _nbytes(ws))
        return
    f = h.shape[1]
    off = None if capacity else group_off
    t, weight = _gemm_types(dtype)
    _call("moe_grouped_gemm_fwd", stream, (x_perm, x_perm_scales, w13, w13_scales, w2, w2_scales, off, gu, h,
                                           y_perm, ws), dtype, weight("x_perm", x_perm, n_rows * d),
          _byte_array("x_perm_scales", x_perm_scales, n_rows * (d // 32)), weight("w13", w13, E * 2 * f * d),
          _byte_array("w13_scales", w13_scales, E * 2 * f * (d // 32)), weight("w2", w2, E * d * f),
          _byte_array("w2_scales", w2_scales, E * d * (f // 32)), _array("group_off", off, _I32, E + 1),
          capacity, E, n_rows, d, f, _array("gu", gu, t, n_rows * 2 * f), _array("h", h, t, n_rows * f),
          _array("y_perm", y_perm, t, n_rows * d), _p(ws), _nbytes(ws))


def moe_grouped_gemm_bwd(dtype, dy_perm, x_perm, gu, h, w13, w2, group_off, capacity, dgu,
                         dx_perm, dw13, dw2, x_perm_scales=None, w13_scales=None, w2_scales=None,
                         ws=None, stream=None):
    """Activation and weight gradients of the grouped SwiGLU FFN (see include/moe.h)."""
    E = group_off.numel() - 1
    n_rows, d = dy_perm.shape
    f = h.shape[1]
    off = None if capacity else group_off
    t, weight = _gemm_types(dtype)
    _call("moe_grouped_gemm_bwd", stream, (dy_perm, x_perm, x_perm_scales, gu, h, w13, w13_scales, w2, w2_scales,
                                           off, dgu, dx_perm, dw13, dw2, ws), dtype,
          _array("dy_perm", dy_perm, t, n_rows * d), weight("x_perm", x_perm, n_rows * d),
          _byte_array("x_perm_scales", x_perm_scales, n_rows * (d // 32)), _array("gu", gu, t, n_rows * 2 * f),
          _array("h", h, t, n_rows * f), weight("w13", w13, E * 2 * f * d),
          _byte_array("w13_scales", w13_scales, E * d * (2 * f // 32)), weight("w2", w2, E * d * f),
          _byte_array("w2_scales", w2_scales, E * f * (d // 32)), _array("group_off", off, _I32, E + 1), capacity,
          E, n_rows, d, f, _array("dgu", dgu, t, n_rows * 2 * f), _array("dx_perm", dx_perm, t, n_rows * d),
          _array("dw13", dw13, t, E * 2 * f * d), _array("dw2", dw2, t, E * d * f), _p(ws), _nbytes(ws))


def gemm_tensors(**tensors):
    """Build a MoeGemmTensors from keyword tensors (names as in GEMM_TENSOR_FIELDS;
    ws is a uint8 workspace tensor whose size becomes ws_bytes)."""
    bad = set(tensors) - set(GEMM_TENSOR_FIELDS) - set(GEMM_TENSOR_FIELDS_F32)
    if bad:
        raise TypeError(f"unknown operand(s) {sorted(bad)}")
    st = MoeGemmTensors(**{n: _p(t) for n, t in tensors.items()})
    if tensors.get("ws") is not None:
        st.ws_bytes = tensors["ws"].numel() * tensors["ws"].element_size()
    st.given = {n: t for n, t in tensors.items() if torch.is_tensor(t)}
    return st


# the operands of each stage
_STAGE = {MOE_GEMM_GATE_UP: ("x_perm", "x_perm_scales", "w13", "w13_scales", "gu", "h"),
          MOE_GEMM_DOWN: ("h", "w2", "w2_scales", "y_perm"),
          MOE_GEMM_DGRAD_DOWN: ("dy_perm", "w2", "w2_scales", "gu", "dgu"),
          MOE_GEMM_DGRAD_GATE_UP: ("dgu", "w13", "w13_scales", "dx_perm"),
          MOE_GEMM_WGRAD: ("dy_perm", "h", "dgu", "x_perm", "x_perm_scales", "dw13", "dw2", "dw13_f32", "dw2_f32")}


def _stage(name, op, dtype, st, group_off, capacity, E, n_rows, d, f, stream, rng, *gate):
    """One stage call, the operands that gemm_tensors() was given checked first."""
    off, key = None if capacity else group_off, (op, dtype, E, n_rows, d, f)
    off_at = _array("group_off", off, _I32, E + 1)
    if st.checked != key:
        st.dev = _check_stage(name, op, dtype, st.given or {}, E, n_rows, d, f)
    dev = st.dev
    for t in (off, rng):
        if torch.is_tensor(t):
            if dev is None:
                dev = t.get_device()
            if t.get_device() != dev or dev < 0:
                raise ValueError(f"{name}: expected tensors on a GPU, all on one, got one on {t.device}")
    args = op, dtype, *gate, ctypes.byref(st), off_at, capacity, E, n_rows, d, f
    _launch(name, torch.cuda.current_device() if dev is None else dev, stream, args)
    st.checked = key


def _check_stage(name, op, dtype, given, E, n_rows, d, f):
    """The GPU of the tensors of `given` that the stage reads and writes (None: there are pointers alone)."""
    size = dict(x_perm=n_rows * d, w13=E * 2 * f * d, w2=E * d * f, gu=n_rows * 2 * f, h=n_rows * f)
    size.update(y_perm=size["x_perm"], dy_perm=size["x_perm"], dx_perm=size["x_perm"], dgu=size["gu"], dw13=size["w13"],
                dw2=size["w2"], dw13_f32=size["w13"], dw2_f32=size["w2"])
    mx, used = dtype in (MOE_MXFP8, MOE_MXFP4), []
    for n in (*_STAGE.get(op, ()), "ws"):
        t = given.get(n)
        if t is None:
            continue
        if n.endswith("_scales"):                           # one of 32 elements
            if mx:
                _byte_array(n, t, size[n[:-7]] // 32)
        elif n.endswith("_f32"):
            _array(n, t, torch.float32, size[n])
        elif mx and n in ("x_perm", "w13", "w2"):
            _byte_array(n, t, size[n] // (2 if dtype == MOE_MXFP4 else 1))
        elif n != "ws" and (mx or dtype in _FLOAT):
            _array(n, t, _FLOAT.get(dtype, torch.bfloat16), size[n])
        used.append(t)
    if not used:
        return None
    dev = used[0].get_device()
    for t in used:
        if t.get_device() != dev or dev < 0:
            raise ValueError(f"{name}: expected tensors on a GPU, all on one, got one on {t.device}")
    return dev


def moe_grouped_gemm_op(op, dtype, tensors, group_off, capacity, E, n_rows, d, f, stream=None):
    """One grouped GEMM stage; tensors is a MoeGemmTensors (gemm_tensors())."""
    _stage("moe_grouped_gemm_op", op, dtype, tensors, group_off, capacity, E, n_rows, d, f, stream, None)


def moe_unpermute_combine(dtype, y_perm, dst_row, weights, k, out, dev_err=None, stream=None):
    """out[t] = sum_j weights[t*k+j] * y_perm[dst_row[t*k+j]] (weights None: unweighted)."""
    T, d = out.shape
    n_rows = y_perm.shape[0]
    t = _float_type(dtype)
    _call("moe_unpermute_combine", stream, (out, y_perm, dst_row, weights, dev_err), dtype,
          _array("y_perm", y_perm, t, n_rows * d), _array("dst_row", dst_row, _I32, T * k),
          _array("weights", weights, torch.float32, T * k), T, k, d, n_rows, _array("out", out, t, T * d),
          _array("dev_err", dev_err, _I32, 1))


def moe_route_add_shared(n_shared, capacity, topk_idx, topk_w, dst_row, counts, offsets, src_slot,
                         topk_idx_out, topk_w_out, counts_out, offsets_out, dst_row_out, src_slot_out,
                         stream=None):
    """The route of k slots -> the route of k + n_shared slots (shared experts E .. E+n_shared-1)."""
    T, k = topk_idx.shape
    E = counts.numel()
    n_rows, K, f32 = src_slot.numel(), k + n_shared, torch.float32
    _call("moe_route_add_shared", stream, (topk_idx, topk_w, dst_row, counts, offsets, src_slot, topk_idx_out, topk_w_out,
                                           counts_out, offsets_out, dst_row_out, src_slot_out), T, E, k, n_shared, capacity,
          _array("topk_idx", topk_idx, _I32, T * k), _array("topk_w", topk_w, f32, T * k),
          _array("dst_row", dst_row, _I32, T * k), _array("counts", counts, _I32, E),
          _array("offsets", offsets, _I32, E + 1), _array("src_slot", src_slot, _I32, 0), n_rows,
          _array("topk_idx_out", topk_idx_out, _I32, T * K), _array("topk_w_out", topk_w_out, f32, T * K),
          _array("counts_out", counts_out, _I32, E + n_shared), _array("offsets_out", offsets_out, _I32, E + n_shared + 1),
          _array("dst_row_out", dst_row_out, _I32, T * K),
          _array("src_slot_out", src_slot_out, _I32, n_rows + n_shared * T))


def moe_router_logits(x, w_router, logits, stream=None):
    """logits [T, E] fp32 = x [T, d] bf16 . w_router [E, d] bf16 ^T."""
    T, d = x.shape
    E = w_router.shape[0]
    _call("moe_router_logits", stream, (x, w_router, logits), _array("x", x, torch.bfloat16, T * d),
          _array("w_router", w_router, torch.bfloat16, E * d), T, E, d, _array("logits", logits, torch.float32, T * E))


def moe_gate_grad(dout, y_perm, topk_idx, topk_w, dst_row, dlogits, dw=None, dy_perm=None,
                  dev_err=None, stream=None):
    """dlogits [T, E] (and optionally dw [T, k], and the combine backward into dy_perm)
    from dout [T, d] and the forward's expert outputs y_perm [n_rows, d]."""
    T, d = dout.shape
    k = topk_idx.shape[1]
    E = dlogits.shape[1]
    n_rows = y_perm.shape[0]
    bf, f32 = torch.bfloat16, torch.float32
    _call("moe_gate_grad", stream, (dout, y_perm, topk_idx, topk_w, dst_row, dlogits, dw, dy_perm, dev_err),
          _array("dout", dout, bf, T * d), _array("y_perm", y_perm, bf, n_rows * d),
          _array("topk_idx", topk_idx, _I32, T * k), _array("topk_w", topk_w, f32, T * k),
          _array("dst_row", dst_row, _I32, T * k), T, E, k, d, n_rows, _array("dlogits", dlogits, f32, T * E),
          _array("dw", dw, f32, T * k), _array("dy_perm", dy_perm, bf, n_rows * d), _array("dev_err", dev_err, _I32, 1))


_FLOAT = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16}


def _float_type(dtype):
    if dtype not in _FLOAT:
        raise MoeError(MOE_EUNSUPPORTED, "a call of fp32 or bf16 tensors")
    return _FLOAT[dtype]


def _rng(rng):
    return _dense("rng", rng, torch.int64, 2)


def moe_dropout(dtype, x, p, rng, out, residual=None, stream=None):
    """out = (residual or 0) + drop(x): fp32 or bf16 tensors of one shape, the mask from rng [2] int64 on the
    device, (seed, step).  The same call on the upstream gradient, without the residual, is the backward."""
    t = _float_type(dtype)
    _call("moe_dropout", stream, (x, residual, rng, out), dtype, _dense("x", x, t, *x.shape),
          _dense("residual", residual, t, *x.shape), x.numel(), p, _rng(rng), _dense("out", out, t, *x.shape))


def moe_combine_dropout(dtype, y_perm, dst_row, weights, k, p, rng, out, residual=None, dev_err=None, stream=None):
    """out[t] = (residual[t] or 0) + drop(sum_j weights[t*k+j] * y_perm[dst_row[t*k+j]]), the mask as
    moe_dropout's over out [T, d]."""
    t = _float_type(dtype)
    T, d = out.shape
    n_rows = y_perm.shape[0]
    if dst_row.numel() != T * k or (weights is not None and weights.numel() != T * k):
        raise ValueError(f"dst_row and weights: expected {T * k} entries for {T} tokens of {k} slots")
    _call("moe_combine_dropout", stream, (out, y_perm, dst_row, weights, residual, rng, dev_err), dtype,
          _dense("y_perm", y_perm, t, n_rows, d), _dense("dst_row", dst_row, torch.int32, *dst_row.shape),
          None if weights is None else _dense("weights", weights, torch.float32, *weights.shape),
          _dense("residual", residual, t, T, d), T, k, d, n_rows, p, _rng(rng), _dense("out", out, t, T, d), _p(dev_err))


def glu(act=MOE_ACT_SILU, limit=0.0, p=0.0, rng=None):
    """A gated block's form: gate MOE_ACT_*, limit on g and u (0: none), dropout of h with probability p and
    rng [2] int64 on the device, (seed, step)."""
    g = MoeGlu(act, limit, p, _rng(rng))
    if limit > 0 and g.limit == 0:
        raise ValueError(f"limit = {limit} is 0 in fp32, which would be no limit")
    g.rng_tensor = rng
    return g


def moe_grouped_glu_op(op, dtype, gate, tensors, group_off, capacity, E, n_rows, d, f, stream=None):
    """One grouped GEMM stage of a gated block of the form gate (glu()); tensors is a MoeGemmTensors."""
    _stage("moe_grouped_glu_op", op, dtype, tensors, group_off, capacity, E, n_rows, d, f, stream, gate.rng_tensor,
           ctypes.byref(gate))


def moe_grouped_glu_fwd(dtype, gate, x_perm, w13, w2, group_off, capacity, gu, h, y_perm, stream=None):
    """moe_grouped_gemm_fwd (fp32, bf16) with the gate, limit and dropout of gate (glu())."""
    t = _float_type(dtype)
    E = group_off.numel() - 1
    n_rows, d = x_perm.shape
    f = w2.shape[-1]
    _call("moe_grouped_glu_fwd", stream, (x_perm, w13, w2, group_off, gu, h, y_perm, gate.rng_tensor), dtype,
          ctypes.byref(gate), _dense("x_perm", x_perm, t, n_rows, d), _dense("w13", w13, t, E, 2 * f, d),
          _dense("w2", w2, t, E, d, f), _dense("group_off", group_off, torch.int32, E + 1), capacity, E, n_rows, d, f,
          _dense("gu", gu, t, n_rows, 2 * f), _dense("h", h, t, n_rows, f), _dense("y_perm", y_perm, t, n_rows, d))


def moe_grouped_glu_bwd(dtype, gate, dy_perm, x_perm, gu, h, w13, w2, group_off, capacity, dgu, dx_perm, dw13, dw2,
                        ws=None, stream=None):
    """moe_grouped_gemm_bwd (fp32, bf16) of moe_grouped_glu_fwd: the same gate, with the rng it had."""
    t = _float_type(dtype)
    E = group_off.numel() - 1
    n_rows, d = dy_perm.shape
    f = w2.shape[-1]
    _call("moe_grouped_glu_bwd", stream, (dy_perm, x_perm, gu, h, w13, w2, group_off, dgu, dx_perm, dw13, dw2, ws,
                                          gate.rng_tensor), dtype, ctypes.byref(gate),
          _dense("dy_perm", dy_perm, t, n_rows, d), _dense("x_perm", x_perm, t, n_rows, d),
          _dense("gu", gu, t, n_rows, 2 * f), _dense("h", h, t, n_rows, f), _dense("w13", w13, t, E, 2 * f, d),
          _dense("w2", w2, t, E, d, f), _dense("group_off", group_off, torch.int32, E + 1), capacity, E, n_rows, d, f,
          _dense("dgu", dgu, t, n_rows, 2 * f), _dense("dx_perm", dx_perm, t, n_rows, d),
          _dense("dw13", dw13, t, E, 2 * f, d), _dense("dw2", dw2, t, E, d, f), _p(ws), _nbytes(ws))


def moe_quantize_int4(src, group, codes, scales, zeros=None, stream=None):
    """bf16 src [rows, K] -> 4-bit codes [rows, K/2] uint8 (element 2i in the low half of byte i), scales
    [rows, K/group] bf16 and, if given, zero points [rows, K/group] uint8."""
    rows, K = src.shape
    _call("moe_quantize_int4", stream, (src, codes, scales, zeros), _dense("src", src, torch.bfloat16, rows, K), rows, K,
          group, _dense("codes", codes, torch.uint8, rows, K // 2),
          _dense("scales", scales, torch.bfloat16, rows, K // group), _dense("zeros", zeros, torch.uint8, rows, K // group))


def moe_dequantize_int4(codes, scales, zeros, group, dst, stream=None):
    """(code - zero) * scale -> dst [rows, K] bf16; zeros None: 8."""
    rows, K = dst.shape
    _call("moe_dequantize_int4", stream, (dst, codes, scales, zeros), _dense("codes", codes, torch.uint8, rows, K // 2),
          _dense("scales", scales, torch.bfloat16, rows, K // group), _dense("zeros", zeros, torch.uint8, rows, K // group),
          rows, K, group, _dense("dst", dst, torch.bfloat16, rows, K))


def moe_int4_workspace_bytes(n_rows, d, f):
    return int(load().moe_int4_workspace_bytes(n_rows, d, f))


def _int4(name, w, E, N, K, group):
    codes, scales, zeros = w
    n = K // group
    return MoeInt4(_dense(name + " codes", codes, torch.uint8, E, N, K // 2),
                   _dense(name + " scales", scales, torch.bfloat16, E, N, n),
                   _dense(name + " zeros", zeros, torch.uint8, E, N, n))


def moe_int4_ffn(gate, x, topk_idx, topk_w, dst_row, src_slot, group_off, group, w13, w2, out, ws, dev_err=None,
                 stream=None):
    """x [T, d] bf16 and the route of its tokens -> out [T, d]: the gated block over experts in 4-bit integers.
    w13 and w2 are (codes, scales, zeros or None) as moe_quantize_int4 makes them: codes [E, 2f, d/2] and
    [E, d, f/2]."""
    T, d = x.shape
    k = topk_idx.shape[1]
    E = group_off.numel() - 1
    f = 2 * w2[0].shape[-1]
    i32 = torch.int32
    if group not in (32, 64, 128):
        raise MoeError(MOE_EUNSUPPORTED, "moe_int4_ffn")
    a, b = _int4("w13", w13, E, 2 * f, d, group), _int4("w2", w2, E, d, f, group)
    if dst_row.numel() != T * k or src_slot.numel() != T * k:
        raise ValueError(f"dst_row and src_slot: expected {T * k} entries for {T} tokens of {k} slots")
    _call("moe_int4_ffn", stream, (x, topk_idx, topk_w, dst_row, src_slot, group_off, *w13, *w2, out, ws, dev_err),
          ctypes.byref(gate), _dense("x", x, torch.bfloat16, T, d), T, k, _dense("topk_idx", topk_idx, i32, T, k),
          _dense("topk_w", topk_w, torch.float32, T, k), _dense("dst_row", dst_row, i32, *dst_row.shape),
          _dense("src_slot", src_slot, i32, *src_slot.shape), _dense("group_off", group_off, i32, E + 1), E, d, f, group,
          ctypes.byref(a), ctypes.byref(b), _dense("out", out, torch.bfloat16, T, d), _p(ws), _nbytes(ws), _p(dev_err))


def moe_quantize_mxfp4(src, codes, scales, stream=None):
    """bf16 src [rows, K] -> E2M1 codes [rows, K/2] (element 2i in the low half of byte i) +
    E8M0 scales [rows, K/32]."""
    rows, K = src.shape
    _call("moe_quantize_mxfp4", stream, (src, codes, scales), _dense("src", src, torch.bfloat16, rows, K), rows, K,
          _dense("codes", codes, torch.uint8, rows, K // 2), _dense("scales", scales, torch.uint8, rows, K // 32))


def moe_dequantize_mxfp4(codes, scales, dst, stream=None):
    """MXFP4 codes [rows, K/2] + scales [rows, K/32] -> their values dst [rows, K] bf16."""
    rows, K = dst.shape
    _call("moe_dequantize_mxfp4", stream, (dst, codes, scales), _dense("codes", codes, torch.uint8, rows, K // 2),
          _dense("scales", scales, torch.uint8, rows, K // 32), rows, K, _dense("dst", dst, torch.bfloat16, rows, K))


def moe_balance_workspace_bytes(T, E, n_seg=1):
    return int(load().moe_balance_workspace_bytes(T, E, n_seg))


def moe_balance_loss(logits, topk_idx, balance_coef, z_coef, losses, counts, probs, lse, tokens, ws,
                     seg_off=None, mask=None, dev_err=None, stream=None):
    """Balance loss and z loss of router logits [T, E] fp32 and topk_idx [T, k] int32 over n_seg
    packed sequences (seg_off [n_seg+1] int32; None: one sequence), tokens with mask [T] uint8 = 0
    left out -> losses [2], counts [n_seg, E] int32, probs [n_seg, E], lse [T] (or None),
    tokens [n_seg+1] int32."""
    T, E = logits.shape
    k = topk_idx.shape[1]
    n_seg = counts.shape[0]
    f32, i32 = torch.float32, torch.int32
    _call("moe_balance_loss", stream, (logits, topk_idx, losses, counts, probs, lse, tokens, ws, seg_off, mask, dev_err),
          _dense("logits", logits, f32, T, E), _dense("topk_idx", topk_idx, i32, T, k),
          _dense("mask", mask, torch.uint8, T), _dense("seg_off", seg_off, i32, n_seg + 1), n_seg, T, E, k,
          balance_coef, z_coef, _dense("losses", losses, f32, 2), _dense("counts", counts, i32, n_seg, E),
          _dense("probs", probs, f32, n_seg, E), _dense("lse", lse, f32, T),
          _dense("tokens", tokens, i32, n_seg + 1), _p(ws), _nbytes(ws), _p(dev_err))


def moe_balance_loss_bwd(logits, counts, tokens, balance_coef, z_coef, dlogits, dlosses=None, add=None,
                         seg_off=None, mask=None, stream=None):
    """dlogits [T, E] = add (or 0) + the gradient of <dlosses, losses> (dlosses [2] on the device,
    None: ones), from counts and tokens as moe_balance_loss wrote them.  add may be dlogits."""
    T, E = logits.shape
    n_seg = counts.shape[0]
    f32, i32 = torch.float32, torch.int32
    _call("moe_balance_loss_bwd", stream, (logits, counts, tokens, dlogits, dlosses, add, seg_off, mask),
          _dense("logits", logits, f32, T, E), _dense("mask", mask, torch.uint8, T),
          _dense("seg_off", seg_off, i32, n_seg + 1), n_seg, T, E, _dense("counts", counts, i32, n_seg, E),
          _dense("tokens", tokens, i32, n_seg + 1), balance_coef, z_coef, _dense("dlosses", dlosses, f32, 2),
          _dense("add", add, f32, T, E), _dense("dlogits", dlogits, f32, T, E))


def moe_quantize_mxfp8(src, colwise, codes, scales, group_off=None, n_groups=0, stream=None):
    """bf16 src [rows, K] -> E4M3FN codes + E8M0 scales (row-wise or per-group column-wise)."""
    rows, K = src.shape
    # column-wise: each group's rows padded to 128
    n = K * (rows + 128 * (n_groups if group_off is not None else 1)) if colwise else rows * K
    _call("moe_quantize_mxfp8", stream, (src, group_off, codes, scales), _array("src", src, torch.bfloat16, rows * K), rows,
          K, int(colwise), _array("group_off", group_off, _I32, n_groups + 1), n_groups, _byte_array("codes", codes, n),
          _byte_array("scales", scales, n // 32))
