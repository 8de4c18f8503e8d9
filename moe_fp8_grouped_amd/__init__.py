"""Python binding of libmoefp8.so, the fp8 MoE grouped-matmul hot path for
MI355X (gfx950).

Argument marshalling only: each function forwards torch tensors' device
pointers, sizes and the current HIP stream to the C entry point of the same
name (declared in include/moe_fp8.h) and raises MoeError on a non-zero
status.  All arithmetic runs in the library's HIP kernels; there is no
fallback path.  The library is built in-tree by ``python -m
moe_fp8_grouped_amd.build``; importing this module without it raises.
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoefp8.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "moe_fp8.h")

# constants mirrored from include/moe_fp8.h
MOE_OK, MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(6)
MOE_DTYPE_DEFAULT, MOE_BF16, MOE_F32, MOE_E4M3FN, MOE_MX4, MOE_E8M0 = -1, 0, 1, 2, 3, 4
MOE_SCALE_ROW_DYNAMIC, MOE_SCALE_TENSOR_DYNAMIC, MOE_SCALE_TENSOR_STATIC = 0, 1, 2
MOE_SCALE_TENSOR_FROM_ROW_AMAX = 3
MOE_ACT_NONE, MOE_ACT_SILU_MUL = 0, 1
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
(MOE_OP_QUANTIZE_ROWS, MOE_OP_SORT_BY_EXPERT, MOE_OP_GMM, MOE_OP_TGMM, MOE_OP_GATHER_REDUCE,
 MOE_OP_QUANTIZE_WEIGHTS, MOE_OP_GMM_MX4, MOE_OP_FFN_TOKENS, MOE_OP_GMM_B128, MOE_OP_TGMM_B128, MOE_OP_BALANCE) = range(11)
MOE_DEVERR_EXPERT_ID, MOE_DEVERR_GROUP_SIZE, MOE_DEVERR_ROWS, MOE_DEVERR_SEQUENCE = 1, 2, 4, 8
MOE_SORT_NOALLOC_SCRATCH_BYTES = 2 << 20

# C signatures: name -> (restype, argtypes)
_P, _I, _I64, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "moe_quantize_rows": (_I, [_P, _P, _I, _I64, _I64, _I, _F, _P, _P, _P, _P, _SZ, _P]),
    "moe_quantize_rows_strided": (_I, [_P, _P, _I64, _I, _I64, _I64, _I, _F, _P, _P, _P, _P, _SZ, _P]),
    "moe_quantize_weights": (_I, [_P, _I64, _I64, _I64, ctypes.c_int32, ctypes.c_int32, _I, _F, _I, _P, _P, _P]),
    "moe_quantize_rows_i8": (_I, [_P, _I64, _I64, _I, _F, _P, _P, _P, _P]),
    "moe_quantize_weights_i8": (_I, [_P, _I64, _I64, _I64, ctypes.c_int32, ctypes.c_int32, _I, _F, _I, _P, _P,
                                     _P]),
    "moe_sort_by_expert": (_I, [_P, _I64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P,
                                _I, _I64, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_sort_by_expert_noalloc": (_I, [_P, _I64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P,
                                        _P, _I, _I64, _I64, _P, _P, _P, _P, _P, _P, _P]),
    "moe_quantize_sort_by_expert": (_I, [_P, _I64, _I64, _I, _F, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                         ctypes.c_int32, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_gmm_fp8": (_I, [_P, _P, _I, _P, _P, ctypes.c_int32, ctypes.c_int32, _I, _P, ctypes.c_int32, ctypes.c_int32,
                         ctypes.c_int32, _I64, _I64, _I64, _I, _P, _P, _SZ, _P]),
    "moe_gmm_i8": (_I, [_P, _P, _I, _P, _P, ctypes.c_int32, ctypes.c_int32, _I, _P, ctypes.c_int32, ctypes.c_int32,
                        ctypes.c_int32, _I64, _I64, _I64, _I, _P, _P, _SZ, _P]),
    "moe_tgmm_fp8": (_I, [_P, _P, ctypes.c_int32, _P, _P, ctypes.c_int32, _P, ctypes.c_int32, ctypes.c_int32,
                          ctypes.c_int32, _I64, _I64, _I64, _I, _P, _P, _SZ, _P]),
    "moe_sort_gather_rows": (_I, [_P, _P, _I, _P, _I64, ctypes.c_int32, _I64, _I64, _P, _P, _P, _SZ, _P]),
    "moe_tgmm_xt_cols": (_I, [_I64, ctypes.c_int32, _P]),
    "moe_sort_gather_transposed": (_I, [_P, _I, _F, _I64, ctypes.c_int32, _I64, _P, _P, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.c_int32, _I64, _P, _P, _P, _SZ, _P]),
    "moe_tgmm_fp8_xt": (_I, [_P, _P, ctypes.c_int32, _P, _P, ctypes.c_int32, _P, ctypes.c_int32, ctypes.c_int32,
                             ctypes.c_int32, _I64, _I64, _I64, _I, _P, _P, _SZ, _P]),
    "moe_gather_reduce": (_I, [_P, _I, _P, _P, _I64, ctypes.c_int32, _I64, _I, _P, _P]),
    "moe_gather_reduce_backward": (_I, [_P, _P, _P, _P, _I64, ctypes.c_int32, _I64, _P, ctypes.c_int32,
                                        ctypes.c_int32, ctypes.c_int32, _I64, _P, _P, _P, _P, _P, _P]),
    "moe_silu_mul_backward": (_I, [_P, _P, _I64, _P, _I64, _I64, _P, _P, _I64, _P]),
    "moe_router_topk": (_I, [_P, _I, _I64, _I64, ctypes.c_int32, ctypes.c_int32, _I, _P, _I, _F, _P, _P, _P]),
    "moe_router_topk_backward": (_I, [_P, _I, _I64, _P, _P, _I64, ctypes.c_int32, ctypes.c_int32, _I, _I, _F, _P, _I64,
                                      _P]),
    "moe_quantize_rows_mx4": (_I, [_P, _P, _I64, _I, _I64, _I64, _P, _I64, _P, _I64, _P]),
    "moe_quantize_weights_mx4": (_I, [_P, _I64, _I64, _I64, _P, _P, _P]),
    "moe_dequantize_rows_mx4": (_I, [_P, _I64, _P, _I64, _I64, _I64, _I, _P, _I64, _P]),
    "moe_gmm_mx4": (_I, [_P, _I64, _P, _I64, _I, _I, _P, _P, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _I64,
                         _I64, _I64, _I, _P, _P, _SZ, _P]),
    "moe_ffn_tokens": (_I, [_P, _I64, _P, _P, _I64, ctypes.c_int32, _I64, _I64, ctypes.c_int32, ctypes.c_int32,
                            ctypes.c_int32, _I, _P, _P, ctypes.c_int32, ctypes.c_int32, _P, _P, ctypes.c_int32,
                            ctypes.c_int32, _I, _P, _P, _SZ, _P]),
    "moe_quantize_rows_b128": (_I, [_P, _P, _I64, _I, _I64, _I64, _P, _I64, _P, _I64, _P]),
    "moe_quantize_weights_b128": (_I, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P]),
    "moe_quantize_cols_b128": (_I, [_P, _P, _I64, _I, _I64, ctypes.c_int32, _P, _P, ctypes.c_int32, ctypes.c_int32,
                                    ctypes.c_int32, _I64, _I64, _P, _P, _P, _SZ, _P]),
    "moe_gmm_b128": (_I, [_P, _I64, _P, _I64, _P, _P, _I, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _I64, _I64,
                          _I64, _I, _P, _P, _SZ, _P]),
    "moe_tgmm_b128": (_I, [_P, _P, _P, _P, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _I64, _I64, _I64, _I, _P, _P,
                           _SZ, _P]),
    "moe_balance_loss": (_I, [_P, _I, _I64, _P, _I64, ctypes.c_int32, ctypes.c_int32, _I, _P, ctypes.c_int32, _P, _P, _P,
                              _P, _SZ, _P]),
    "moe_balance_loss_backward": (_I, [_P, _I, _I64, _P, _P, _P, _I64, ctypes.c_int32, ctypes.c_int32, _I, _P,
                                       ctypes.c_int32, _I, _P, _I64, _P]),
    "moe_workspace_bytes": (_I, [_I, _I64, _I64, _I64, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_debug_check": (_I, [_P, _P, ctypes.POINTER(ctypes.c_int32)]),
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_version": (_I, []),
}


class MoeError(RuntimeError):
    def __init__(self, fn, status, text):
        super().__init__(f"{fn} failed with status {status}: {text}")
        self.status = status


_lib = None


def load_library(path=LIB_PATH):
    """dlopen libmoefp8.so and attach the C signatures (no GPU needed)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libmoefp8.so is not built ({path}); run python -m moe_fp8_grouped_amd.build")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor or None")
    if not t.is_cuda:
        raise ValueError("tensor arguments must live in GPU memory")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return t.data_ptr()


_current_device = torch.cuda.current_device
# the handle alone: 0.2 us, where building torch's stream object around it takes 2.7
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _current_handle is None:
            return torch.cuda.current_stream().cuda_stream
        return _current_handle(_current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _stream_here(stream, *tensors):
    """_stream, for tensors (and a stream) that must belong to the current device, where the kernels are launched."""
    here = _current_device()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError("tensor arguments must live on the current device (%d)" % here)
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != here:
        raise ValueError("the stream must belong to the current device (%d)" % here)
    return _stream(stream)


def _call(name, *args):
    st = getattr(load_library(), name)(*args)
    if st != MOE_OK:
        raise MoeError(name, st, status_string(st))
    return st


def status_string(status):
    return load_library().moe_status_string(status).decode()


def version():
    return load_library().moe_version()


def workspace_bytes(op, d0=0, d1=0, d2=0, E=1):
    out = ctypes.c_size_t(0)
    st = load_library().moe_workspace_bytes(op, d0, d1, d2, E, ctypes.byref(out))
    if st != MOE_OK:
        raise MoeError("moe_workspace_bytes", st, status_string(st))
    return out.value


def workspace(op, d0=0, d1=0, d2=0, E=1, device="cuda"):
    """A zeroed workspace tensor (uint8) of the size the library asks for."""
    return torch.zeros(workspace_bytes(op, d0, d1, d2, E), dtype=torch.uint8, device=device)


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def moe_quantize_rows(x, x_up, act, R, C, scale_mode, static_scale, q, scale, row_amax=None, ws=None, stream=None):
    return _call("moe_quantize_rows", _ptr(x), _ptr(x_up), act, R, C, scale_mode, float(static_scale), _ptr(q),
                 _ptr(scale), _ptr(row_amax), _ptr(ws), _nbytes(ws), _stream(stream))


def _ptr_rows(t, ld):
    """Device pointer of a 2-D view whose rows are ``ld`` elements apart (unit inner stride)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("tensor arguments must be torch tensors in GPU memory")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (shape[1] > 1 and stride[1] != 1) or (shape[0] > 1 and stride[0] != ld):
        raise ValueError("expected a 2-D view with rows %d elements apart" % ld)
    return t.data_ptr()


def moe_quantize_rows_strided(x, x_up, ldx, act, R, C, scale_mode, static_scale, q, scale, row_amax=None, ws=None,
                              stream=None):
    return _call("moe_quantize_rows_strided", _ptr_rows(x, ldx), _ptr_rows(x_up, ldx), ldx, act, R, C, scale_mode,
                 float(static_scale), _ptr(q), _ptr(scale), _ptr(row_amax), _ptr(ws), _nbytes(ws), _stream(stream))


def moe_quantize_weights(w, E, K, N, kb, nb, scale_mode, static_scale, transpose_out, q, scale, stream=None):
    return _call("moe_quantize_weights", _ptr(w), E, K, N, kb, nb, scale_mode, float(static_scale),
                 transpose_out, _ptr(q), _ptr(scale), _stream(stream))


def moe_quantize_rows_i8(x, R, C, scale_mode, static_scale, q, scale, row_amax=None, stream=None):
    return _call("moe_quantize_rows_i8", _ptr(x), R, C, scale_mode, float(static_scale), _ptr(q), _ptr(scale),
                 _ptr(row_amax), _stream(stream))


def moe_quantize_weights_i8(w, E, K, N, kb, nb, scale_mode, static_scale, transpose_out, q, scale, stream=None):
    return _call("moe_quantize_weights_i8", _ptr(w), E, K, N, kb, nb, scale_mode, float(static_scale),
                 transpose_out, _ptr(q), _ptr(scale), _stream(stream))


def moe_sort_by_expert(expert_ids, T, k, E, group_offset, num_local_experts, xq, xscale, xscale_mode, H, M_cap,
                       perm, inv_pos, group_sizes, xs, ss, ws, stream=None):
    return _call("moe_sort_by_expert", _ptr(expert_ids), T, k, E, group_offset, num_local_experts, _ptr(xq),
                 _ptr(xscale), xscale_mode, H, M_cap, _ptr(perm), _ptr(inv_pos), _ptr(group_sizes), _ptr(xs),
                 _ptr(ss), _ptr(ws), _nbytes(ws), _stream(stream))


def moe_sort_by_expert_noalloc(expert_ids, T, k, E, group_offset, num_local_experts, xq, xscale, xscale_mode, H,
                               M_cap, perm, inv_pos, group_sizes, xs, ss, device_error=None, stream=None):
    return _call("moe_sort_by_expert_noalloc", _ptr(expert_ids), T, k, E, group_offset, num_local_experts, _ptr(xq),
                 _ptr(xscale), xscale_mode, H, M_cap, _ptr(perm), _ptr(inv_pos), _ptr(group_sizes), _ptr(xs),
                 _ptr(ss), _ptr(device_error), _stream(stream))


def moe_quantize_sort_by_expert(x, T, H, scale_mode, static_scale, expert_ids, k, E, group_offset, num_local_experts,
                                M_cap, perm, inv_pos, group_sizes, xs, ss, scale=None, ws=None, stream=None,
                                row_amax=None):
    return _call("moe_quantize_sort_by_expert", _ptr(x), T, H, scale_mode, float(static_scale), _ptr(expert_ids), k,
                 E, group_offset, num_local_experts, M_cap, _ptr(perm), _ptr(inv_pos), _ptr(group_sizes), _ptr(xs),
                 _ptr(ss), _ptr(scale), _ptr(row_amax), _ptr(ws), _nbytes(ws), _stream(stream))


def moe_gmm_fp8(lhs, lhs_scale, lhs_scale_mode, rhs, rhs_scale, Kb, Nb, transpose_rhs, group_sizes, E,
                group_offset, num_local_experts, M, K, N, out_dtype, out, ws, stream=None):
    return _call("moe_gmm_fp8", _ptr(lhs), _ptr(lhs_scale), lhs_scale_mode, _ptr(rhs), _ptr(rhs_scale), Kb, Nb,
                 transpose_rhs, _ptr(group_sizes), E, group_offset, num_local_experts, M, K, N, out_dtype,
                 _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream))


def moe_gmm_i8(lhs, lhs_scale, lhs_scale_mode, rhs, rhs_scale, Kb, Nb, transpose_rhs, group_sizes, E,
               group_offset, num_local_experts, M, K, N, out_dtype, out, ws, stream=None):
    return _call("moe_gmm_i8", _ptr(lhs), _ptr(lhs_scale), lhs_scale_mode, _ptr(rhs), _ptr(rhs_scale), Kb, Nb,
                 transpose_rhs, _ptr(group_sizes), E, group_offset, num_local_experts, M, K, N, out_dtype,
                 _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream))


def moe_tgmm_fp8(lhs, lhs_scale, lhs_scale_len, rhs, rhs_scale, rhs_scale_len, group_sizes, E, group_offset,
                 num_local_experts, M, K, N, out_dtype, out, ws, stream=None):
    return _call("moe_tgmm_fp8", _ptr(lhs), _ptr(lhs_scale), lhs_scale_len, _ptr(rhs), _ptr(rhs_scale),
                 rhs_scale_len, _ptr(group_sizes), E, group_offset, num_local_experts, M, K, N, out_dtype,
                 _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream))


def moe_sort_gather_rows(xq, xscale, xscale_mode, inv_pos, T, k, H, M_cap, xs, ss, ws, stream=None):
    return _call("moe_sort_gather_rows", _ptr(xq), _ptr(xscale), xscale_mode, _ptr(inv_pos), T, k, H, M_cap,
                 _ptr(xs), _ptr(ss), _ptr(ws), _nbytes(ws), _stream(stream))


def tgmm_xt_cols(M, E):
    out = ctypes.c_int64(0)
    st = load_library().moe_tgmm_xt_cols(M, E, ctypes.byref(out))
    if st != MOE_OK:
        raise MoeError("moe_tgmm_xt_cols", st, status_string(st))
    return out.value


def moe_sort_gather_transposed(x, x_dtype, static_scale, T, k, H, perm, group_sizes, E, group_offset,
                               num_local_experts, M, xt, scale_out, ws, stream=None):
    return _call("moe_sort_gather_transposed", _ptr(x), x_dtype, float(static_scale), T, k, H, _ptr(perm),
                 _ptr(group_sizes), E, group_offset, num_local_experts, M, _ptr(xt), _ptr(scale_out), _ptr(ws),
                 _nbytes(ws), _stream(stream))


def moe_tgmm_fp8_xt(xt, lhs_scale, lhs_scale_len, rhs, rhs_scale, rhs_scale_len, group_sizes, E, group_offset,
                    num_local_experts, M, K, N, out_dtype, out, ws, stream=None):
    return _call("moe_tgmm_fp8_xt", _ptr(xt), _ptr(lhs_scale), lhs_scale_len, _ptr(rhs), _ptr(rhs_scale),
                 rhs_scale_len, _ptr(group_sizes), E, group_offset, num_local_experts, M, K, N, out_dtype,
                 _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream))


def moe_gather_reduce(y, y_dtype, inv_pos, topk_weights, T, k, N, out_dtype, out, stream=None):
    return _call("moe_gather_reduce", _ptr(y), y_dtype, _ptr(inv_pos), _ptr(topk_weights), T, k, N, out_dtype,
                 _ptr(out), _stream(stream))


def moe_gather_reduce_backward(dout, y, inv_pos, topk_weights, T, k, N, group_sizes, E, group_offset,
                               num_local_experts, M_cap, dy, dw, dy_q=None, dy_scale=None, dy_amax=None, stream=None):
    return _call("moe_gather_reduce_backward", _ptr(dout), _ptr(y), _ptr(inv_pos), _ptr(topk_weights), T, k, N,
                 _ptr(group_sizes), E, group_offset, num_local_experts, M_cap, _ptr(dy), _ptr(dw), _ptr(dy_q),
                 _ptr(dy_scale), _ptr(dy_amax), _stream(stream))


def moe_silu_mul_backward(a, b, lda, dh, R, C, da, db, ldo, stream=None):
    """a, b, da, db may be column slices of wider buffers (row strides lda, ldo)."""
    return _call("moe_silu_mul_backward", _ptr_rows(a, lda), _ptr_rows(b, lda), lda, _ptr(dh), R, C,
                 _ptr_rows(da, ldo), _ptr_rows(db, ldo), ldo, _stream(stream))


def moe_router_topk(logits, logits_dtype, ldl, T, E, k, score, select_bias, renormalize, weight_scale, expert_ids,
                    topk_weights, stream=None):
    """logits may be a column slice of a wider buffer (row stride ldl)."""
    return _call("moe_router_topk", _ptr_rows(logits, ldl), logits_dtype, ldl, T, E, k, score, _ptr(select_bias),
                 renormalize, float(weight_scale), _ptr(expert_ids), _ptr(topk_weights),
                 _stream_here(stream, logits, select_bias, expert_ids, topk_weights))


def moe_router_topk_backward(logits, logits_dtype, ldl, expert_ids, dweights, T, E, k, score, renormalize, weight_scale,
                             dlogits, ldd, stream=None):
    """logits and dlogits may be column slices of wider buffers (row strides ldl, ldd)."""
    return _call("moe_router_topk_backward", _ptr_rows(logits, ldl), logits_dtype, ldl, _ptr(expert_ids),
                 _ptr(dweights), T, E, k, score, renormalize, float(weight_scale), _ptr_rows(dlogits, ldd), ldd,
                 _stream_here(stream, logits, expert_ids, dweights, dlogits))


def moe_quantize_rows_mx4(x, x_up, ldx, act, R, C, q, ldq, scale, lds, stream=None):
    """x, x_up, q, scale may be column slices of wider buffers (row strides ldx, ldx, ldq, lds)."""
    return _call("moe_quantize_rows_mx4", _ptr_rows(x, ldx), _ptr_rows(x_up, ldx), ldx, act, R, C, _ptr_rows(q, ldq), ldq,
                 _ptr_rows(scale, lds), lds, _stream_here(stream, x, x_up, q, scale))


def moe_quantize_weights_mx4(w, E, K, N, q, scale, stream=None):
    return _call("moe_quantize_weights_mx4", _ptr(w), E, K, N, _ptr(q), _ptr(scale), _stream_here(stream, w, q, scale))


def moe_dequantize_rows_mx4(q, ldq, scale, lds, R, C, out_dtype, out, ldo, stream=None):
    """q, scale, out may be column slices of wider buffers (row strides ldq, lds, ldo)."""
    return _call("moe_dequantize_rows_mx4", _ptr_rows(q, ldq), ldq, _ptr_rows(scale, lds), lds, R, C, out_dtype,
                 _ptr_rows(out, ldo), ldo, _stream_here(stream, q, scale, out))


def moe_gmm_mx4(lhs, ldl, lhs_scale, lds, lhs_format, lhs_scale_mode, rhs, rhs_scale, group_sizes, E, group_offset,
                num_local_experts, M, K, N, out_dtype, out, ws, stream=None):
    """lhs, and with MOE_MX4 its scales, may be column slices of wider buffers (row strides ldl, lds)."""
    ls = _ptr_rows(lhs_scale, lds) if lhs_format == MOE_MX4 else _ptr(lhs_scale)
    return _call("moe_gmm_mx4", _ptr_rows(lhs, ldl), ldl, ls, lds, lhs_format, lhs_scale_mode, _ptr(rhs), _ptr(rhs_scale),
                 _ptr(group_sizes), E, group_offset, num_local_experts, M, K, N, out_dtype, _ptr(out), _ptr(ws),
                 _nbytes(ws), _stream_here(stream, lhs, lhs_scale, rhs, rhs_scale, group_sizes, out, ws))


def moe_ffn_tokens(x, ldx, expert_ids, topk_weights, T, k, H, I, E, group_offset, num_local_experts, w_format, w01,
                   w01_scale, kb01, nb01, wo, wo_scale, kbo, nbo, out_dtype, out, ws, stream=None):
    """x may be a column slice of a wider buffer (row stride ldx)."""
    return _call("moe_ffn_tokens", _ptr_rows(x, ldx), ldx, _ptr(expert_ids), _ptr(topk_weights), T, k, H, I, E,
                 group_offset, num_local_experts, w_format, _ptr(w01), _ptr(w01_scale), kb01, nb01, _ptr(wo),
                 _ptr(wo_scale), kbo, nbo, out_dtype, _ptr(out), _ptr(ws), _nbytes(ws),
                 _stream_here(stream, x, expert_ids, topk_weights, w01, w01_scale, wo, wo_scale, out, ws))


def moe_quantize_rows_b128(x, x_up, ldx, act, R, C, q, ldq, scale, lds, stream=None):
    """x, x_up, q, scale may be column slices of wider buffers (row strides ldx, ldx, ldq, lds)."""
    return _call("moe_quantize_rows_b128", _ptr_rows(x, ldx), _ptr_rows(x_up, ldx), ldx, act, R, C, _ptr_rows(q, ldq), ldq,
                 _ptr_rows(scale, lds), lds, _stream_here(stream, x, x_up, q, scale))


def moe_quantize_weights_b128(w, E, K, N, q, scale, qt=None, scale_t=None, stream=None):
    return _call("moe_quantize_weights_b128", _ptr(w), E, K, N, _ptr(q), _ptr(scale), _ptr(qt), _ptr(scale_t),
                 _stream_here(stream, w, q, scale, qt, scale_t))


def moe_quantize_cols_b128(x, x_up, ldx, act, T, k, perm, group_sizes, E, group_offset, num_local_experts, M, C, qt, scale_t,
                           ws, stream=None):
    """x, x_up may be column slices of wider buffers (row stride ldx)."""
    return _call("moe_quantize_cols_b128", _ptr_rows(x, ldx), _ptr_rows(x_up, ldx), ldx, act, T, k, _ptr(perm),
                 _ptr(group_sizes), E, group_offset, num_local_experts, M, C, _ptr(qt), _ptr(scale_t), _ptr(ws), _nbytes(ws),
                 _stream_here(stream, x, x_up, perm, group_sizes, qt, scale_t, ws))


def moe_gmm_b128(lhs, ldl, lhs_scale, lds, rhs, rhs_scale, rhs_scale_dtype, group_sizes, E, group_offset, num_local_experts,
                 M, K, N, out_dtype, out, ws, stream=None):
    """lhs and its scales may be column slices of wider buffers (row strides ldl, lds)."""
    return _call("moe_gmm_b128", _ptr_rows(lhs, ldl), ldl, _ptr_rows(lhs_scale, lds), lds, _ptr(rhs), _ptr(rhs_scale),
                 rhs_scale_dtype, _ptr(group_sizes), E, group_offset, num_local_experts, M, K, N, out_dtype, _ptr(out),
                 _ptr(ws), _nbytes(ws), _stream_here(stream, lhs, lhs_scale, rhs, rhs_scale, group_sizes, out, ws))


def moe_tgmm_b128(lhs_t, lhs_scale, rhs_t, rhs_scale, group_sizes, E, group_offset, num_local_experts, M, K, N, out_dtype, out,
                  ws, stream=None):
    return _call("moe_tgmm_b128", _ptr(lhs_t), _ptr(lhs_scale), _ptr(rhs_t), _ptr(rhs_scale), _ptr(group_sizes), E,
                 group_offset, num_local_experts, M, K, N, out_dtype, _ptr(out), _ptr(ws), _nbytes(ws),
                 _stream_here(stream, lhs_t, lhs_scale, rhs_t, rhs_scale, group_sizes, out, ws))


def moe_balance_loss(logits, logits_dtype, ldl, expert_ids, T, E, k, score, seq_offsets, S, loss, counts, tokens, ws,
                     stream=None):
    """logits may be a column slice of a wider buffer (row stride ldl)."""
    return _call("moe_balance_loss", _ptr_rows(logits, ldl), logits_dtype, ldl, _ptr(expert_ids), T, E, k, score,
                 _ptr(seq_offsets), S, _ptr(loss), _ptr(counts), _ptr(tokens), _ptr(ws), _nbytes(ws),
                 _stream_here(stream, logits, expert_ids, seq_offsets, loss, counts, tokens, ws))


def moe_balance_loss_backward(logits, logits_dtype, ldl, counts, tokens, dloss, T, E, k, score, seq_offsets, S, accumulate,
                              dlogits, ldd, stream=None):
    """logits and dlogits may be column slices of wider buffers (row strides ldl, ldd)."""
    return _call("moe_balance_loss_backward", _ptr_rows(logits, ldl), logits_dtype, ldl, _ptr(counts), _ptr(tokens),
                 _ptr(dloss), T, E, k, score, _ptr(seq_offsets), S, accumulate, _ptr_rows(dlogits, ldd), ldd,
                 _stream_here(stream, logits, counts, tokens, dloss, seq_offsets, dlogits))


def moe_debug_check(ws, stream=None):
    """Synchronise and return the sticky device-error word of a workspace."""
    err = ctypes.c_int32(0)
    st = load_library().moe_debug_check(_ptr(ws), _stream(stream), ctypes.byref(err))
    if st != MOE_OK:
        raise MoeError("moe_debug_check", st, status_string(st))
    return err.value
