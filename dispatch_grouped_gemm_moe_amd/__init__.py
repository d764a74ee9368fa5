"""Python binding of the MI355X fused MoE layer library (include/moe.h).

Argument marshalling only: every entry point below forwards torch tensors'
device pointers and the caller's current HIP stream to the C ABI function of
the same name in ``_lib/libmoe_mi355x.so``.  All computation happens in the
library's HIP kernels; there is no CPU or PyTorch fallback.  Importing this
package fails loudly if the library has not been built
(``python -m dispatch_grouped_gemm_moe_amd.build``).
"""
from __future__ import annotations

import array
import ctypes
import dataclasses
import operator
import os

from .build import lib_path

MOE_OK, MOE_E_INVALID, MOE_E_UNSUPPORTED, MOE_E_WORKSPACE, MOE_E_HIP, MOE_E_DEVICE = range(6)
MOE_PREC_BF16, MOE_PREC_MXFP8 = 0, 1
MOE_F_SHARED_EXPERT = 1 << 0
MOE_F_IDENTITY_EXPERTS = 1 << 1
MOE_F_LAUNCH_PER_GEMM = 1 << 2
MOE_F_DEBUG_DROP_SIGNAL = 1 << 3
MOE_F_BF16_WGRAD = 1 << 4
MOE_DEV_OK, MOE_DEV_WAIT_TIMEOUT = 0, 1

# every symbol include/moe.h declares
EXPORTS = ("moe_status_string", "moe_abi_version", "moe_validate_cfg", "moe_query_sizes",
           "moe_prepare_weights", "moe_route", "moe_dispatch_layout", "moe_layer_fwd",
           "moe_layer_bwd", "moe_read_device_status", "moe_mx_quantize", "moe_timing_enable",
           "moe_timing_read", "moe_diag_mfma_loop", "moe_layer_fwd_static", "moe_mx_dequantize",
           "moe_add_rmsnorm_fwd", "moe_add_rmsnorm_bwd", "moe_query_add_rmsnorm_bwd", "moe_layer_fwd_few",
           "moe_query_few", "moe_dispatch_rows", "moe_combine_rows", "moe_combine_rows_bwd", "moe_block_quantize",
           "moe_block_quantize_weights", "moe_block_dequantize", "moe_block_gemm", "moe_query_block_swiglu",
           "moe_block_gemm_swiglu", "moe_query_grad_norm", "moe_grad_norm", "moe_clip_grads")
MOE_STATIC_WORKSPACE_BYTES = 256 << 20
MOE_FEW_MAX_TOKENS, MOE_FEW_COUNTER_BYTES = 64, 36864
MOE_GRAD_COUNTER_BYTES = 8448
KERNEL_KINDS = ("route", "layout", "gemm_gate_up", "gemm_down", "combine", "gather", "other", "wgrad",
                "dgrad_down", "dgrad_gate_up", "shared_gemm", "layer")


class moe_cfg(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("minibatch", ctypes.c_int32),
                ("ring_slots", ctypes.c_int32), ("comm_cus", ctypes.c_int32),
                ("prec", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class moe_sizes(ctypes.Structure):
    _fields_ = [("packed_weights", ctypes.c_size_t), ("workspace_fwd", ctypes.c_size_t),
                ("saved", ctypes.c_size_t), ("workspace_bwd", ctypes.c_size_t),
                ("minibatch", ctypes.c_int32), ("ring_slots", ctypes.c_int32),
                ("num_minibatches", ctypes.c_int32), ("comm_cus", ctypes.c_int32)]


class moe_weights(ctypes.Structure):
    _fields_ = [("Wr", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("packed", ctypes.c_void_p),
                ("packed_bytes", ctypes.c_size_t)]


class moe_kernel_times(ctypes.Structure):
    _fields_ = [("launches", ctypes.c_int32 * 12), ("ms", ctypes.c_double * 12), ("dropped", ctypes.c_int32)]


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__("%s: %s (status %d)" % (fn, _load().moe_status_string(status).decode(), status))


_LIB = None


def _load():
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise ImportError("HIP library %s is missing: build it with "
                              "`python -m dispatch_grouped_gemm_moe_amd.build`" % path)
        lib = ctypes.CDLL(path)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        cfgp = ctypes.POINTER(moe_cfg)
        sig = {
            "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "moe_abi_version": (I32, []),
            "moe_validate_cfg": (ctypes.c_int, [cfgp]),
            "moe_query_sizes": (ctypes.c_int, [cfgp, ctypes.POINTER(moe_sizes)]),
            "moe_prepare_weights": (ctypes.c_int, [cfgp, P, P, P, P, P, P, P, SZ, P]),
            "moe_route": (ctypes.c_int, [cfgp, P, P, P, P, P, P, P, P, P]),
            "moe_dispatch_layout": (ctypes.c_int, [cfgp, P, P, P, P, P, P]),
            "moe_layer_fwd": (ctypes.c_int, [cfgp, ctypes.POINTER(moe_weights), P, P, P, SZ, P, SZ, P]),
            "moe_layer_bwd": (ctypes.c_int, [cfgp, ctypes.POINTER(moe_weights), P, P, P, SZ, P, P, P,
                                             P, P, P, P, P, SZ, P]),
            "moe_read_device_status": (ctypes.c_int, [P, P, ctypes.POINTER(I32), ctypes.POINTER(I32)]),
            "moe_mx_quantize": (ctypes.c_int, [P, ctypes.c_int64, I32, P, P, P]),
            "moe_timing_enable": (ctypes.c_int, [I32]),
            "moe_timing_read": (ctypes.c_int, [ctypes.POINTER(moe_kernel_times)]),
            "moe_diag_mfma_loop": (ctypes.c_int, [I32, P, ctypes.c_int64, I32, I32, P, P, P]),
            "moe_layer_fwd_static": (ctypes.c_int, [cfgp, ctypes.POINTER(moe_weights), P, P, P, P]),
            "moe_mx_dequantize": (ctypes.c_int, [P, P, ctypes.c_int64, I32, I32, P, P]),
            "moe_add_rmsnorm_fwd": (ctypes.c_int, [ctypes.c_int64, I32, P, P, P, ctypes.c_float, P, P, P, P, P, P, P,
                                                   P]),
            "moe_query_add_rmsnorm_bwd": (ctypes.c_int, [ctypes.c_int64, I32, ctypes.POINTER(SZ)]),
            "moe_add_rmsnorm_bwd": (ctypes.c_int, [ctypes.c_int64, I32, P, P, P, P, P, P, P, P, P, P, SZ, P]),
            "moe_layer_fwd_few": (ctypes.c_int, [cfgp, ctypes.POINTER(moe_weights), P, P, P, P, P, SZ, P]),
            "moe_query_few": (ctypes.c_int, [cfgp, ctypes.POINTER(SZ)]),
            "moe_dispatch_rows": (ctypes.c_int, [I64, I32, I32, I64, P, P, P, P, P, P]),
            "moe_combine_rows": (ctypes.c_int, [I64, I32, I32, I64, P, P, P, P, P, P]),
            "moe_combine_rows_bwd": (ctypes.c_int, [I64, I32, I32, I64, P, P, P, P, P, P, P, P, P]),
            "moe_block_quantize": (ctypes.c_int, [I64, I32, P, P, P, P]),
            "moe_block_quantize_weights": (ctypes.c_int, [I32, I32, I32, P, I32, P, P, P]),
            "moe_block_dequantize": (ctypes.c_int, [I64, I32, I32, P, P, P, P]),
            "moe_block_gemm": (ctypes.c_int, [I64, I32, I32, I32, P, P, P, P, P, P, P]),
            "moe_query_block_swiglu": (ctypes.c_int, [I64, I32, I32, I32, ctypes.POINTER(SZ)]),
            "moe_block_gemm_swiglu": (ctypes.c_int, [I64, I32, I32, I32, P, P, P, P, P, P, P, P, P, P, P, SZ, P]),
            "moe_query_grad_norm": (ctypes.c_int, [I32, ctypes.POINTER(SZ)]),
            "moe_grad_norm": (ctypes.c_int, [I32, P, P, P, P, P, SZ, P]),
            "moe_clip_grads": (ctypes.c_int, [I32, P, P, P, P, ctypes.c_float, P, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(lib, name)
            f.restype, f.argtypes = res, args
        _LIB = lib
    return _LIB


def lib():
    """The loaded ctypes library (loads it on first use)."""
    return _load()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    return ctypes.c_void_p(stream if isinstance(stream, int) else stream.cuda_stream)


def _check(fn, st):
    if st != MOE_OK:
        raise MoeError(fn, st)


def make_cfg(T, H, I, E, k, minibatch=0, ring_slots=0, comm_cus=0, prec=MOE_PREC_BF16, flags=0) -> moe_cfg:
    return moe_cfg(T, H, I, E, k, minibatch, ring_slots, comm_cus, prec, flags)


# ---------------------------------------------------------------- entry points

def moe_abi_version() -> int:
    return _load().moe_abi_version()


def moe_validate_cfg(cfg: moe_cfg) -> int:
    return _load().moe_validate_cfg(ctypes.byref(cfg))


def moe_query_sizes(cfg: moe_cfg) -> moe_sizes:
    s = moe_sizes()
    _check("moe_query_sizes", _load().moe_query_sizes(ctypes.byref(cfg), ctypes.byref(s)))
    return s


def moe_prepare_weights(cfg, Wg, Wu, Wd, packed, Wsg=None, Wsu=None, Wsd=None, stream=None):
    _check("moe_prepare_weights", _load().moe_prepare_weights(
        ctypes.byref(cfg), _ptr(Wg), _ptr(Wu), _ptr(Wd), _ptr(Wsg), _ptr(Wsu), _ptr(Wsd),
        _ptr(packed), packed.numel() * packed.element_size(), _stream(stream)))


def moe_route(cfg, x, Wr, bias, topk_idx, topk_w, logits=None, x_codes=None, x_scales=None, stream=None):
    _check("moe_route", _load().moe_route(ctypes.byref(cfg), _ptr(x), _ptr(Wr), _ptr(bias),
                                          _ptr(topk_idx), _ptr(topk_w), _ptr(logits), _ptr(x_codes),
                                          _ptr(x_scales), _stream(stream)))


def moe_dispatch_layout(cfg, topk_idx, counts, offsets, row_token, tok_row, stream=None):
    _check("moe_dispatch_layout", _load().moe_dispatch_layout(
        ctypes.byref(cfg), _ptr(topk_idx), _ptr(counts), _ptr(offsets), _ptr(row_token),
        _ptr(tok_row), _stream(stream)))


def _weights(Wr, bias, packed) -> moe_weights:
    return moe_weights(Wr.data_ptr(), bias.data_ptr() if bias is not None else None,
                       packed.data_ptr(), packed.numel() * packed.element_size())


def moe_layer_fwd(cfg, Wr, bias, packed, x, out, ws, saved=None, stream=None):
    w = _weights(Wr, bias, packed)
    _check("moe_layer_fwd", _load().moe_layer_fwd(
        ctypes.byref(cfg), ctypes.byref(w), _ptr(x), _ptr(out), _ptr(saved),
        0 if saved is None else saved.numel() * saved.element_size(), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def moe_layer_fwd_static(cfg, Wr, bias, packed, x, out, status=None, stream=None):
    """Forward on the library's static workspace (allocates nothing); status: an
    int32 device tensor of 2 elements that receives the device status word."""
    w = _weights(Wr, bias, packed)
    _check("moe_layer_fwd_static", _load().moe_layer_fwd_static(
        ctypes.byref(cfg), ctypes.byref(w), _ptr(x), _ptr(out), _ptr(status), _stream(stream)))


def moe_layer_bwd(cfg, Wr, bias, packed, x, dout, saved, dx, dWg, dWu, dWd, dWr, ws,
                  dWs=None, dgate=None, stream=None):
    w = _weights(Wr, bias, packed)
    _check("moe_layer_bwd", _load().moe_layer_bwd(
        ctypes.byref(cfg), ctypes.byref(w), _ptr(x), _ptr(dout), _ptr(saved),
        saved.numel() * saved.element_size(), _ptr(dx), _ptr(dWg), _ptr(dWu), _ptr(dWd), _ptr(dWr),
        _ptr(dWs), _ptr(dgate), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_read_device_status(ws, stream=None):
    code, detail = ctypes.c_int32(0), ctypes.c_int32(0)
    st = _load().moe_read_device_status(_ptr(ws), _stream(stream), ctypes.byref(code), ctypes.byref(detail))
    return st, code.value, detail.value


def _sizes(fn, rows, cols):
    """rows and cols, refused where the int64 and int32 of the C call cannot hold them: ctypes would pass
    their low bits on."""
    if not (-1 << 31 <= cols < 1 << 31 and -1 << 63 <= rows < 1 << 63):
        raise MoeError(fn, MOE_E_UNSUPPORTED)
    return rows, cols


def moe_mx_quantize(src, codes, scales, stream=None):
    rows, cols = _sizes("moe_mx_quantize", *src.shape)
    _check("moe_mx_quantize", _load().moe_mx_quantize(_ptr(src), rows, cols, _ptr(codes), _ptr(scales),
                                                      _stream(stream)))


_dtype = operator.attrgetter("dtype")
torch = None  # until a call is given tensors: building, sizing and validating need none


def _use_torch():
    """torch, and its tensors' methods as functions: looked up once, not for each of a call's tensors."""
    global torch, _numel, _is_contiguous, _get_device, _data_ptr, _GRAD_KINDS, _CODE_KINDS
    import torch
    _CODE_KINDS = torch.uint8, torch.float8_e4m3fn
    _GRAD_KINDS = {torch.float32: 0, torch.bfloat16: 1}
    _numel, _is_contiguous = torch.Tensor.numel, torch.Tensor.is_contiguous
    _get_device, _data_ptr = torch.Tensor.get_device, torch.Tensor.data_ptr


def _dense(fn, device, t, dtype, n):
    """The pointer of a dense tensor of `dtype` with at least n elements on `device` (its index, -1 for
    the host); None stays None.  The kernels see pointers only, so what they could not read is refused
    here."""
    if t is None:
        return None
    if t.dtype is not dtype or _numel(t) < n or not _is_contiguous(t) or _get_device(t) != device:
        raise MoeError(fn, MOE_E_INVALID)
    return _data_ptr(t)


def _buffer(fn, device, t):
    """The pointer and the bytes of a dense buffer on `device`, a tensor of any type."""
    if not _is_contiguous(t) or _get_device(t) != device:
        raise MoeError(fn, MOE_E_INVALID)
    return _data_ptr(t), t.nbytes


def _call(fn, device, stream, *args):
    """Library function fn(*args, stream) on `device`: the given stream, or that device's current one.  A
    launch goes to the current device's queues, so that one is made current for the call.  Host tensors
    are refused: the kernels would fault on them."""
    if device < 0:
        raise MoeError(fn, MOE_E_INVALID)
    if device == torch._C._cuda_getDevice():
        if stream is None:
            s = torch._C._cuda_getCurrentRawStream(device)
        else:
            s = stream if isinstance(stream, int) else stream.cuda_stream
        st = getattr(_load(), fn)(*args, s)
        if st != MOE_OK:
            raise MoeError(fn, st)
    else:
        with torch.cuda.device(device):
            _call(fn, device, stream, *args)


def moe_mx_dequantize(codes, scales, dst, operand_scales=False, stream=None):
    """dst (bf16) = the values of codes [rows, cols] and their scales: [rows, cols/32], or with
    operand_scales the GEMM operand layout [ceil(cols/128), rows, 4]."""
    if torch is None:
        _use_torch()
    fn, dev, u8 = "moe_mx_dequantize", codes.get_device(), torch.uint8
    rows, cols = _sizes(fn, *codes.shape)
    n_scales = (cols + 127) // 128 * rows * 4 if operand_scales else rows * (cols // 32)
    _call(fn, dev, stream, _dense(fn, dev, codes, u8, 0), _dense(fn, dev, scales, u8, n_scales), rows, cols,
          1 if operand_scales else 0, _dense(fn, dev, dst, torch.bfloat16, rows * cols))


def moe_add_rmsnorm_fwd(x, weight, y, eps=1e-6, residual=None, summed=None, rstd=None, y_codes=None, y_scales=None,
                        ck_codes=None, ck_scales=None, stream=None):
    """y = rmsnorm(x + residual) * weight over the rows of x [rows, cols]; see include/moe.h for the
    optional outputs (the sum, 1/rms, the MXFP8 form of y, the 8-bit checkpoint of the sum)."""
    if torch is None:
        _use_torch()
    fn, dev, b16, f32, u8 = "moe_add_rmsnorm_fwd", x.get_device(), torch.bfloat16, torch.float32, torch.uint8
    rows, cols = _sizes(fn, *x.shape)
    n = rows * cols
    _call(fn, dev, stream, rows, cols, _dense(fn, dev, x, b16, n), _dense(fn, dev, residual, b16, n),
          _dense(fn, dev, weight, f32, cols), eps, _dense(fn, dev, summed, b16, n), _dense(fn, dev, y, b16, n),
          _dense(fn, dev, rstd, f32, rows), _dense(fn, dev, y_codes, u8, n),
          _dense(fn, dev, y_scales, u8, (cols + 127) // 128 * rows * 4), _dense(fn, dev, ck_codes, u8, n),
          _dense(fn, dev, ck_scales, u8, rows * (cols // 32)))


def moe_query_add_rmsnorm_bwd(rows, cols) -> int:
    fn, n = "moe_query_add_rmsnorm_bwd", ctypes.c_size_t()
    _check(fn, _load().moe_query_add_rmsnorm_bwd(*_sizes(fn, rows, cols), ctypes.byref(n)))
    return n.value


def moe_add_rmsnorm_bwd(dy, weight, rstd, dx, dweight, ws, summed=None, ck_codes=None, ck_scales=None, dsum=None,
                        stream=None):
    """dx and dweight of moe_add_rmsnorm_fwd, from the sum or from its 8-bit checkpoint."""
    if torch is None:
        _use_torch()
    fn, dev, b16, f32, u8 = "moe_add_rmsnorm_bwd", dy.get_device(), torch.bfloat16, torch.float32, torch.uint8
    rows, cols = _sizes(fn, *dy.shape)
    n = rows * cols
    _call(fn, dev, stream, rows, cols, _dense(fn, dev, dy, b16, n), _dense(fn, dev, dsum, b16, n),
          _dense(fn, dev, summed, b16, n), _dense(fn, dev, ck_codes, u8, n),
          _dense(fn, dev, ck_scales, u8, rows * (cols // 32)), _dense(fn, dev, weight, f32, cols),
          _dense(fn, dev, rstd, f32, rows), _dense(fn, dev, dx, b16, n), _dense(fn, dev, dweight, f32, cols),
          *_buffer(fn, dev, ws))


def moe_query_few(cfg: moe_cfg) -> int:
    n = ctypes.c_size_t()
    _check("moe_query_few", _load().moe_query_few(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def moe_layer_fwd_few(cfg, Wr, bias, packed, x, out, ws, x_codes=None, x_scales=None, stream=None):
    """Layer forward for cfg.T <= MOE_FEW_MAX_TOKENS tokens; ws: moe_query_few bytes, the first
    MOE_FEW_COUNTER_BYTES of them zeroed once."""
    if torch is None:
        _use_torch()
    fn, dev, b16, f32, u8 = "moe_layer_fwd_few", x.get_device(), torch.bfloat16, torch.float32, torch.uint8
    T, H, E = cfg.T, cfg.H, cfg.E
    w = moe_weights(_dense(fn, dev, Wr, f32, H * E), _dense(fn, dev, bias, f32, E), *_buffer(fn, dev, packed))
    _call(fn, dev, stream, ctypes.byref(cfg), ctypes.byref(w), _dense(fn, dev, x, b16, T * H),
          _dense(fn, dev, x_codes, u8, T * H), _dense(fn, dev, x_scales, u8, (H + 127) // 128 * T * 4),
          _dense(fn, dev, out, b16, T * H), *_buffer(fn, dev, ws))


def _blocks(n):
    return (n + 127) // 128


def _codes(fn, device, t, n):
    """_dense of E4M3 codes: as bytes, or in torch's own type for them, in which a checkpoint's arrive."""
    if t is None:
        return None
    if t.dtype not in _CODE_KINDS or _numel(t) < n or not _is_contiguous(t) or _get_device(t) != device:
        raise MoeError(fn, MOE_E_INVALID)
    return _data_ptr(t)


def _row_scales(fn, device, t, rows, cols):
    """The pointer of the scales [ceil(cols / 128), rows] of rows in blocks of 128.  A matrix of more columns
    would be read in another order: refused."""
    if t is not None and t.dim() > 1 and t.shape[-1] != rows:
        raise MoeError(fn, MOE_E_INVALID)
    return _dense(fn, device, t, torch.float32, _blocks(cols) * rows)


def moe_dispatch_rows(x, tok_row, dst=None, codes=None, scales=None, stream=None):
    """Row tok_row[t, j] = x[t] for each of the k choices j: of dst (bf16), and / or of codes and scales
    (moe_block_quantize's); rows outside theirs are no rows."""
    if torch is None:
        _use_torch()
    fn, dev, b16 = "moe_dispatch_rows", x.get_device(), torch.bfloat16
    T, cols = _sizes(fn, *x.shape)
    k = tok_row.shape[1]
    R = dst.shape[0] if dst is not None else codes.shape[0] if codes is not None else 0
    if codes is not None and codes.shape[0] != R:
        raise MoeError(fn, MOE_E_INVALID)
    _call(fn, dev, stream, T, k, cols, R, _dense(fn, dev, x, b16, 0), _dense(fn, dev, tok_row, torch.int32, T * k),
          _dense(fn, dev, dst, b16, R * cols), _codes(fn, dev, codes, R * cols),
          _row_scales(fn, dev, scales, R, cols))


def moe_combine_rows(src, tok_row, out, topk_w=None, add=None, stream=None):
    """out[t] = add[t] + sum over j of topk_w[t, j] src[tok_row[t, j]]; without topk_w the weights are 1,
    which is the gradient of moe_dispatch_rows."""
    if torch is None:
        _use_torch()
    fn, dev, b16, f32 = "moe_combine_rows", src.get_device(), torch.bfloat16, torch.float32
    R, cols = _sizes(fn, *src.shape)
    T, k = tok_row.shape
    _call(fn, dev, stream, T, k, cols, R, _dense(fn, dev, src, b16, 0), _dense(fn, dev, tok_row, torch.int32, 0),
          _dense(fn, dev, topk_w, f32, T * k), _dense(fn, dev, add, b16, T * cols), _dense(fn, dev, out, b16, T * cols))


def moe_combine_rows_bwd(dout, tok_row, src=None, topk_w=None, dsrc=None, dw=None, codes=None, scales=None,
                         stream=None):
    """dsrc[tok_row[t, j]] = topk_w[t, j] dout[t] (bf16, and / or its codes and scales) and
    dw[t, j] = <src[tok_row[t, j]], dout[t]>."""
    if torch is None:
        _use_torch()
    fn, dev, b16, f32 = "moe_combine_rows_bwd", dout.get_device(), torch.bfloat16, torch.float32
    T, cols = _sizes(fn, *dout.shape)
    k = tok_row.shape[1]
    rows = {t.shape[0] for t in (src, dsrc, codes) if t is not None}
    if len(rows) > 1:
        raise MoeError(fn, MOE_E_INVALID)
    R = rows.pop() if rows else 0
    _call(fn, dev, stream, T, k, cols, R, _dense(fn, dev, dout, b16, 0), _dense(fn, dev, src, b16, R * cols),
          _dense(fn, dev, tok_row, torch.int32, T * k), _dense(fn, dev, topk_w, f32, T * k),
          _dense(fn, dev, dsrc, b16, R * cols), _codes(fn, dev, codes, R * cols),
          _row_scales(fn, dev, scales, R, cols), _dense(fn, dev, dw, f32, T * k))


def moe_block_quantize(src, codes, scales, stream=None):
    """codes [rows, cols] and scales [ceil(cols / 128), rows] of src (bf16) in blocks of 1 x 128."""
    if torch is None:
        _use_torch()
    fn, dev = "moe_block_quantize", src.get_device()
    rows, cols = _sizes(fn, *src.shape)
    _call(fn, dev, stream, rows, cols, _dense(fn, dev, src, torch.bfloat16, 0),
          _codes(fn, dev, codes, rows * cols), _row_scales(fn, dev, scales, rows, cols))


def moe_block_quantize_weights(src, codes, scales, transposed=False, stream=None):
    """codes [groups, n, k] and scales [groups, ceil(n / 128), ceil(k / 128)] in blocks of 128 x 128 of src
    (bf16) [groups, n, k], or with transposed [groups, k, n]."""
    if torch is None:
        _use_torch()
    fn, dev = "moe_block_quantize_weights", src.get_device()
    groups, n, k = codes.shape
    if max(groups, n, k) >= 1 << 31:
        raise MoeError(fn, MOE_E_UNSUPPORTED)
    _call(fn, dev, stream, groups, n, k, _dense(fn, dev, src, torch.bfloat16, groups * n * k), 1 if transposed else 0,
          _codes(fn, dev, codes, 0), _dense(fn, dev, scales, torch.float32, groups * _blocks(n) * _blocks(k)))


def moe_block_dequantize(codes, scales, dst, weights=False, stream=None):
    """dst (bf16) = the values of codes [rows, cols] and their scales, or with weights of codes [groups, n, k]."""
    if torch is None:
        _use_torch()
    fn, dev = "moe_block_dequantize", codes.get_device()
    n = codes.shape[-2] if weights else 0
    rows, cols = _sizes(fn, codes.shape[0] * n if weights else codes.shape[0], codes.shape[-1])
    if n >= 1 << 31:
        raise MoeError(fn, MOE_E_UNSUPPORTED)
    s = _dense(fn, dev, scales, torch.float32, codes.shape[0] * _blocks(n) * _blocks(cols)) if weights else \
        _row_scales(fn, dev, scales, rows, cols)
    _call(fn, dev, stream, rows, cols, n, _codes(fn, dev, codes, rows * cols), s,
          _dense(fn, dev, dst, torch.bfloat16, rows * cols))


def _block_operands(fn, dev, a, a_scales, offsets, w):
    """The sizes of a product and the pointers of its rows: (rows, n, k, groups), (a, a_scales, offsets)."""
    rows, k = _sizes(fn, *a.shape)
    groups, n, kw = w.shape
    if kw != k:
        raise MoeError(fn, MOE_E_INVALID)
    if max(groups, n) >= 1 << 31:
        raise MoeError(fn, MOE_E_UNSUPPORTED)
    return (rows, n, k, groups), (_codes(fn, dev, a, 0), _row_scales(fn, dev, a_scales, rows, k),
                                  _dense(fn, dev, offsets, torch.int32, groups + 1))


def moe_block_gemm(a, a_scales, w, w_scales, out, offsets=None, stream=None):
    """out [rows, n] (bf16) = rows of a [rows, k] times their group's matrix w [groups, n, k], both codes in
    blocks of 128 with their scales; group g's rows are offsets[g] .. offsets[g + 1] - 1."""
    if torch is None:
        _use_torch()
    fn, dev = "moe_block_gemm", a.get_device()
    (rows, n, k, groups), ptrs = _block_operands(fn, dev, a, a_scales, offsets, w)
    _call(fn, dev, stream, rows, n, k, groups, *ptrs, _codes(fn, dev, w, 0),
          _dense(fn, dev, w_scales, torch.float32, groups * _blocks(n) * _blocks(k)),
          _dense(fn, dev, out, torch.bfloat16, rows * n))


def moe_query_block_swiglu(rows, n, k, groups) -> int:
    """Bytes of moe_block_gemm_swiglu's workspace for so many rows or fewer."""
    fn, size = "moe_query_block_swiglu", ctypes.c_size_t()
    for v in n, k, groups:
        _sizes(fn, rows, v)
    _check(fn, _load().moe_query_block_swiglu(rows, n, k, groups, ctypes.byref(size)))
    return size.value


def moe_block_gemm_swiglu(a, a_scales, wg, wg_scales, wu, wu_scales, h_codes, h_scales, ws, h=None, offsets=None,
                          stream=None):
    """h = silu(a wg) * (a wu), each as moe_block_gemm's product, in codes h_codes [rows, n] and scales h_scales
    [ceil(n / 128), rows], and in bf16 where h is given; ws: moe_query_block_swiglu bytes."""
    if torch is None:
        _use_torch()
    fn, dev, f32 = "moe_block_gemm_swiglu", a.get_device(), torch.float32
    (rows, n, k, groups), ptrs = _block_operands(fn, dev, a, a_scales, offsets, wg)
    if wu.shape != wg.shape:
        raise MoeError(fn, MOE_E_INVALID)
    n_s = groups * _blocks(n) * _blocks(k)
    _call(fn, dev, stream, rows, n, k, groups, *ptrs, _codes(fn, dev, wg, 0), _dense(fn, dev, wg_scales, f32, n_s),
          _codes(fn, dev, wu, 0), _dense(fn, dev, wu_scales, f32, n_s), _codes(fn, dev, h_codes, rows * n),
          _row_scales(fn, dev, h_scales, rows, n), _dense(fn, dev, h, torch.bfloat16, rows * n),
          *_buffer(fn, dev, ws))


def moe_query_grad_norm(tensors) -> int:
    """Bytes of moe_grad_norm's workspace for so many tensors; its first MOE_GRAD_COUNTER_BYTES are zeroed once."""
    fn, n = "moe_query_grad_norm", ctypes.c_size_t()
    if not 0 <= tensors < 1 << 31:
        raise MoeError(fn, MOE_E_INVALID)
    _check(fn, _load().moe_query_grad_norm(tensors, ctypes.byref(n)))
    return n.value


def _grad_arrays(fn, dev, grads):
    """Arrays of the tensors' pointers, element counts and types (1: bf16), as the C calls read them."""
    if not all(map(_is_contiguous, grads)) or set(map(_get_device, grads)) - {dev}:
        raise MoeError(fn, MOE_E_INVALID)
    try:
        kinds = bytes(map(_GRAD_KINDS.__getitem__, map(_dtype, grads)))
    except KeyError:
        raise MoeError(fn, MOE_E_INVALID) from None
    return array.array("Q", list(map(_data_ptr, grads))), array.array("q", list(map(_numel, grads))), kinds


def _address(a):
    return a.buffer_info()[0]


def moe_grad_norm(grads, norm, ws, stream=None):
    """norm (one fp32 element) = the norm of all tensors' (fp32 or bf16) elements together; ws:
    moe_query_grad_norm bytes, the first MOE_GRAD_COUNTER_BYTES of them zeroed once."""
    if torch is None:
        _use_torch()
    fn, dev = "moe_grad_norm", norm.get_device()
    ptrs, counts, kinds = _grad_arrays(fn, dev, grads)
    _call(fn, dev, stream, len(kinds), _address(ptrs), _address(counts), kinds, _dense(fn, dev, norm, torch.float32, 1),
          *_buffer(fn, dev, ws))


def moe_clip_grads(grads, norm, max_norm, out=None, stream=None):
    """out[i] = grads[i] * min(1, max_norm / (norm + 1e-6)), in place without out; norm as moe_grad_norm wrote it."""
    if torch is None:
        _use_torch()
    fn, dev = "moe_clip_grads", norm.get_device()
    ptrs, counts, kinds = _grad_arrays(fn, dev, grads)
    outs = ptrs
    if out is not None:
        outs, *like = _grad_arrays(fn, dev, out)
        if like != [counts, kinds]:  # other sizes or types
            raise MoeError(fn, MOE_E_INVALID)
    _call(fn, dev, stream, len(kinds), _address(ptrs), _address(counts), kinds, _dense(fn, dev, norm, torch.float32, 1),
          max_norm, _address(outs))


def moe_diag_mfma_loop(kind, operands, blocks, iters, clocks, sink, stream=None):
    """Sustained-MFMA diagnostic: kind 0 = bf16, 1 = MXFP8 (E4M3 codes); operands
    >= 16 KiB, clocks int64 [2], sink fp32 [blocks*512]."""
    _check("moe_diag_mfma_loop", _load().moe_diag_mfma_loop(kind, _ptr(operands),
                                                            operands.numel() * operands.element_size(), blocks,
                                                            iters, _ptr(clocks), _ptr(sink), _stream(stream)))


def moe_timing_enable(on: bool):
    _check("moe_timing_enable", _load().moe_timing_enable(1 if on else 0))


def moe_timing_read() -> dict:
    """{kind: (launches, total_ms)} since the last moe_timing_enable(True)."""
    t = moe_kernel_times()
    _check("moe_timing_read", _load().moe_timing_read(ctypes.byref(t)))
    res = {n: (t.launches[i], t.ms[i]) for i, n in enumerate(KERNEL_KINDS)}
    res["dropped"] = t.dropped
    return res


# ---------------------------------------------------------------- buffers

@dataclasses.dataclass
class LayerBuffers:
    """Device buffers of one layer configuration, allocated with torch."""

    cfg: moe_cfg
    sizes: moe_sizes
    packed: object
    ws: object
    saved: object | None


def alloc_buffers(cfg: moe_cfg, device="cuda", with_saved=False) -> LayerBuffers:
    import torch
    s = moe_query_sizes(cfg)
    packed = torch.empty(s.packed_weights, dtype=torch.uint8, device=device)
    ws = torch.zeros(max(s.workspace_fwd, s.workspace_bwd) if with_saved else s.workspace_fwd,
                     dtype=torch.uint8, device=device)
    saved = torch.empty(s.saved, dtype=torch.uint8, device=device) if with_saved else None
    return LayerBuffers(cfg, s, packed, ws, saved)
