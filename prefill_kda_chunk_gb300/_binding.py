"""ctypes binding of libkda_gb300.so (include/kda.h).

Argument marshalling only: every step of the prefill runs in the library's
CUDA kernels. PyTorch supplies device memory and the current stream. There
is no fallback: if the library is missing or the device is not sm_103, calls
raise.

`stream` of a call is a raw handle, for programs that order their streams
themselves: the tensors that the call makes belong to PyTorch's current stream, and
their memory may still be in use there. Give such a call its outputs, or make its
stream the current one.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libkda_gb300.so")

STATUS = {
    0: "KDA_OK", -1: "KDA_ERR_NULL_ARG", -2: "KDA_ERR_BAD_SHAPE", -3: "KDA_ERR_UNSUPPORTED_DIM",
    -4: "KDA_ERR_MISALIGNED", -5: "KDA_ERR_BAD_CU_SEQLENS", -6: "KDA_ERR_CUDA",
    -7: "KDA_ERR_DEVICE_TIMEOUT", -8: "KDA_ERR_NO_DEVICE_SUPPORT", -9: "KDA_ERR_ALIAS",
    -10: "KDA_ERR_GATE_RANGE", -11: "KDA_ERR_CAPTURE", -12: "KDA_ERR_WRONG_DEVICE",
    -13: "KDA_ERR_NOT_DEVICE_MEMORY", -14: "KDA_ERR_SCRATCH_LIMIT", -15: "KDA_ERR_BAD_FLAGS",
    -16: "KDA_ERR_BAD_PAGE_TABLE", -17: "KDA_ERR_OUT_OF_PAGES",
}
# input preprocessing flags (include/kda.h)
PRE_NORM_QK = 1
PRE_GATE_LOGITS = 2
# flags of the short convolution and of the state space scan
CONV_SILU = 1
CONV_DOUT_FP32 = 2
SSM_DT_SOFTPLUS = 1
# flags of the norms with the rotation
ROPE_INTERLEAVED = 1
ROPE_DOUT_FP32 = 2
STATUS_CODE = {v: k for k, v in STATUS.items()}

_lib = None
_lock = threading.Lock()


class KdaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        self.name = STATUS.get(code, str(code))
        super().__init__(f"{where}: {self.name} ({kda_status_string(code)})")


def lib() -> ctypes.CDLL:
    """Load the library (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(
                    f"{LIB_PATH} is missing; build it with "
                    "`python -m prefill_kda_chunk_gb300.build`")
            L = ctypes.CDLL(LIB_PATH)
            vp, i64, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float
            L.kda_chunk_prefill.restype = ctypes.c_int
            L.kda_chunk_prefill.argtypes = [vp] * 7 + [i64] * 6 + [f32, vp, vp, vp]
            L.kda_chunk_prefill_ex.restype = ctypes.c_int
            L.kda_chunk_prefill_ex.argtypes = [vp] * 7 + [i64] * 6 + [f32, ctypes.c_int, vp, vp, vp]
            L.kda_chunk_prefill_noalloc.restype = ctypes.c_int
            L.kda_chunk_prefill_noalloc.argtypes = [vp] * 7 + [i64] * 6 + [f32, vp, vp, vp]
            L.kda_decode_step.restype = ctypes.c_int
            L.kda_decode_step.argtypes = [vp] * 7 + [i64] * 4 + [f32, ctypes.c_int, vp, vp]
            L.kda_backward_workspace_bytes.restype = ctypes.c_int64
            L.kda_backward_workspace_bytes.argtypes = [i64] * 4 + [ctypes.c_int]
            L.kda_chunk_prefill_backward.restype = ctypes.c_int
            L.kda_chunk_prefill_backward.argtypes = [vp] * 7 + [i64] * 6 + [f32] + [vp] * 9
            L.kda_short_conv.restype = ctypes.c_int
            L.kda_short_conv.argtypes = [vp] * 5 + [i64] * 6 + [ctypes.c_int, vp, i64, vp, vp]
            L.kda_short_conv_step.restype = ctypes.c_int
            L.kda_short_conv_step.argtypes = [vp] * 4 + [i64] * 4 + [ctypes.c_int, vp, i64, vp, vp]
            L.kda_short_conv_backward.restype = ctypes.c_int
            L.kda_short_conv_backward.argtypes = ([vp] * 5 + [i64] * 6 + [ctypes.c_int, vp, i64, vp,
                                                  vp, i64] + [vp] * 4)
            L.kda_test_conv_backward_plan.restype = ctypes.c_int
            L.kda_test_conv_backward_plan.argtypes = ([vp] * 3 + [i64] * 6
                                                      + [ctypes.c_int, ctypes.POINTER(i64)])
            L.kda_ssm_prefill.restype = ctypes.c_int
            L.kda_ssm_prefill.argtypes = [vp] * 9 + [i64] * 11 + [ctypes.c_int, vp, vp, vp]
            L.kda_ssm_step.restype = ctypes.c_int
            L.kda_ssm_step.argtypes = [vp] * 8 + [i64] * 9 + [ctypes.c_int, vp, vp, vp]
            L.kda_paged_decode.restype = ctypes.c_int
            L.kda_paged_decode.argtypes = [vp] * 5 + [i64] * 9 + [f32, vp, vp, vp]
            L.kda_page_plan.restype = ctypes.c_int
            L.kda_page_plan.argtypes = [vp] * 6 + [i64] * 5 + [vp] * 8
            L.kda_qk_norm_rope.restype = ctypes.c_int
            L.kda_qk_norm_rope.argtypes = ([vp] * 6 + [i64] * 7 + [f32, ctypes.c_int, vp, i64, vp, i64,
                                           vp])
            L.kda_qk_norm_rope_backward.restype = ctypes.c_int
            L.kda_qk_norm_rope_backward.argtypes = ([vp] * 6 + [i64] * 7 + [f32, ctypes.c_int]
                                                    + [vp, i64] * 4 + [vp] * 3)
            L.kda_paged_append_fp8.restype = ctypes.c_int
            L.kda_paged_append_fp8.argtypes = [vp] * 9 + [i64] * 17 + [vp]
            L.kda_paged_decode_fp8.restype = ctypes.c_int
            L.kda_paged_decode_fp8.argtypes = [vp] * 7 + [i64] * 15 + [f32, vp, vp, vp]
            L.kda_status_string.restype = ctypes.c_char_p
            L.kda_status_string.argtypes = [ctypes.c_int]
            L.kda_last_device_error.restype = ctypes.c_int
            L.kda_last_device_error.argtypes = [vp]
            L.kda_workspace_release.restype = ctypes.c_int
            L.kda_workspace_release.argtypes = []
            L.kda_workspace_bytes.restype = i64
            L.kda_workspace_bytes.argtypes = [i64, i64, i64, i64, ctypes.c_int]
            L.kda_stage_timing_begin.restype = ctypes.c_int
            L.kda_stage_timing_begin.argtypes = [ctypes.c_int]
            L.kda_stage_timing_end.restype = ctypes.c_int
            L.kda_stage_timing_end.argtypes = [ctypes.POINTER(ctypes.c_double),
                                               ctypes.POINTER(ctypes.c_double),
                                               ctypes.POINTER(ctypes.c_int)]
            L.kda_set_recurrent_impl.restype = ctypes.c_int
            L.kda_set_recurrent_impl.argtypes = [ctypes.c_int]
            L.kda_set_scan_segments.restype = ctypes.c_int
            L.kda_set_scan_segments.argtypes = [ctypes.c_int]
            L.kda_set_backward_impl.restype = ctypes.c_int
            L.kda_set_backward_impl.argtypes = [ctypes.c_int]
            L.kda_test_stall_recurrent.restype = ctypes.c_int
            L.kda_test_stall_recurrent.argtypes = [ctypes.c_int, i64]
            L.kda_test_stall_scan.restype = ctypes.c_int
            L.kda_test_stall_scan.argtypes = [ctypes.c_int]
            L.kda_test_stall_qk_norm_rope.restype = ctypes.c_int
            L.kda_test_stall_qk_norm_rope.argtypes = [ctypes.c_int]
            L.kda_test_stall_paged_fp8.restype = ctypes.c_int
            L.kda_test_stall_paged_fp8.argtypes = [ctypes.c_int]
            L.kda_build_info.restype = ctypes.c_char_p
            L.kda_build_info.argtypes = []
            _lib = L
    return _lib


# ------------------------------------------------------------ raw C calls

def kda_chunk_prefill(q, k, v, g, beta, initial_state, cu_seqlens, B, T, H, K, V, N, scale,
                      out, final_state, stream) -> int:
    """The C entry point, pointers as ints (0 = NULL). Returns the status."""
    return lib().kda_chunk_prefill(q, k, v, g, beta, initial_state, cu_seqlens, B, T, H, K, V, N,
                                   scale, out, final_state, stream)


def kda_chunk_prefill_ex(q, k, v, g, beta, initial_state, cu_seqlens, B, T, H, K, V, N, scale,
                         flags, out, final_state, stream) -> int:
    """The C entry point with input preprocessing flags (PRE_*)."""
    return lib().kda_chunk_prefill_ex(q, k, v, g, beta, initial_state, cu_seqlens, B, T, H, K, V,
                                      N, scale, flags, out, final_state, stream)


def kda_chunk_prefill_noalloc(q, k, v, g, beta, initial_state, cu_seqlens, B, T, H, K, V, N,
                              scale, out, final_state, stream) -> int:
    """The allocation-free C entry point (fixed 64 MiB scratch inside the
    library), pointers as ints. Returns the status."""
    return lib().kda_chunk_prefill_noalloc(q, k, v, g, beta, initial_state, cu_seqlens, B, T, H,
                                           K, V, N, scale, out, final_state, stream)


def kda_decode_step(q, k, v, g, beta, state_in, state_out, N, H, K, V, scale, flags, out,
                    stream) -> int:
    """The one-token decode C entry point, pointers as ints (0 = NULL)."""
    return lib().kda_decode_step(q, k, v, g, beta, state_in, state_out, N, H, K, V, scale, flags,
                                 out, stream)


def kda_backward_workspace_bytes(B, T, H, N, has_cu_seqlens) -> int:
    """Workspace bytes of a gradient call with these sizes (0 on bad sizes)."""
    return lib().kda_backward_workspace_bytes(B, T, H, N, int(bool(has_cu_seqlens)))


def kda_chunk_prefill_backward(q, k, v, g, beta, initial_state, cu_seqlens, B, T, H, K, V, N,
                               scale, d_out, d_final_state, dq, dk, dv, dg, dbeta,
                               d_initial_state, stream) -> int:
    """The gradient C entry point, pointers as ints (0 = NULL)."""
    return lib().kda_chunk_prefill_backward(q, k, v, g, beta, initial_state, cu_seqlens, B, T, H,
                                            K, V, N, scale, d_out, d_final_state, dq, dk, dv, dg,
                                            dbeta, d_initial_state, stream)


def kda_short_conv(x, weight, bias, initial_state, cu_seqlens, B, T, D, W, N, x_stride, flags,
                   out, out_stride, final_state, stream) -> int:
    """The short-convolution C entry point, pointers as ints (0 = NULL)."""
    return lib().kda_short_conv(x, weight, bias, initial_state, cu_seqlens, B, T, D, W, N,
                                x_stride, flags, out, out_stride, final_state, stream)


def kda_short_conv_step(x, weight, bias, state_in, N, D, W, x_stride, flags, out, out_stride,
                        state_out, stream) -> int:
    """The single-token convolution C entry point, pointers as ints (0 = NULL)."""
    return lib().kda_short_conv_step(x, weight, bias, state_in, N, D, W, x_stride, flags, out,
                                     out_stride, state_out, stream)


def kda_short_conv_backward(x, weight, bias, initial_state, cu_seqlens, B, T, D, W, N, x_stride,
                            flags, d_out, dout_stride, d_final_state, dx, dx_stride, dweight,
                            dbias, d_initial_state, stream) -> int:
    """The convolution's gradient C entry point, pointers as ints (0 = NULL)."""
    return lib().kda_short_conv_backward(x, weight, bias, initial_state, cu_seqlens, B, T, D, W,
                                         N, x_stride, flags, d_out, dout_stride, d_final_state,
                                         dx, dx_stride, dweight, dbias, d_initial_state, stream)


def kda_ssm_prefill(x, dt, a, b, c, d, dt_bias, initial_state, cu_seqlens, B, T, H, P, G, n, N,
                    x_stride, dt_stride, b_stride, c_stride, flags, out, final_state,
                    stream) -> int:
    """The state space scan C entry point, pointers as ints (0 = NULL)."""
    return lib().kda_ssm_prefill(x, dt, a, b, c, d, dt_bias, initial_state, cu_seqlens, B, T, H,
                                 P, G, n, N, x_stride, dt_stride, b_stride, c_stride, flags, out,
                                 final_state, stream)


def kda_ssm_step(x, dt, a, b, c, d, dt_bias, state_in, N, H, P, G, n, x_stride, dt_stride,
                 b_stride, c_stride, flags, out, state_out, stream) -> int:
    """The single-token scan C entry point, pointers as ints (0 = NULL)."""
    return lib().kda_ssm_step(x, dt, a, b, c, d, dt_bias, state_in, N, H, P, G, n, x_stride,
                              dt_stride, b_stride, c_stride, flags, out, state_out, stream)


def kda_paged_decode(q, k_cache, v_cache, page_table, seq_lens, B, Hq, Hkv, D, pages, page_size,
                     max_pages, k_page_stride, v_page_stride, scale, out, lse, stream) -> int:
    """The paged decode attention C entry point, pointers as ints (0 = NULL)."""
    return lib().kda_paged_decode(q, k_cache, v_cache, page_table, seq_lens, B, Hq, Hkv, D, pages,
                                  page_size, max_pages, k_page_stride, v_page_stride, scale, out,
                                  lse, stream)


def kda_page_plan(page_table, seq_lens, new_lens, release, free_pages, free_count, B, max_pages, pool,
                  page_size, T, page_table_out, seq_lens_out, free_pages_out, free_count_out,
                  cu_seqlens, positions, slots, stream) -> int:
    """The page plan C entry point, pointers as ints (0 = NULL)."""
    return lib().kda_page_plan(page_table, seq_lens, new_lens, release, free_pages, free_count, B,
                               max_pages, pool, page_size, T, page_table_out, seq_lens_out,
                               free_pages_out, free_count_out, cu_seqlens, positions, slots, stream)


def kda_qk_norm_rope(q, k, q_weight, k_weight, inv_freq, positions, T, Hq, Hk, D, R, q_stride, k_stride,
                     eps, flags, q_out, q_out_stride, k_out, k_out_stride, stream) -> int:
    """The C entry point of the norms with the rotation, pointers as ints (0 = NULL)."""
    return lib().kda_qk_norm_rope(q, k, q_weight, k_weight, inv_freq, positions, T, Hq, Hk, D, R,
                                  q_stride, k_stride, eps, flags, q_out, q_out_stride, k_out,
                                  k_out_stride, stream)


def kda_qk_norm_rope_backward(q, k, q_weight, k_weight, inv_freq, positions, T, Hq, Hk, D, R, q_stride,
                              k_stride, eps, flags, dq_out, dq_out_stride, dk_out, dk_out_stride, dq,
                              dq_stride, dk, dk_stride, dq_weight, dk_weight, stream) -> int:
    """The C entry point of their gradients, pointers as ints (0 = NULL)."""
    return lib().kda_qk_norm_rope_backward(q, k, q_weight, k_weight, inv_freq, positions, T, Hq, Hk, D,
                                           R, q_stride, k_stride, eps, flags, dq_out, dq_out_stride,
                                           dk_out, dk_out_stride, dq, dq_stride, dk, dk_stride,
                                           dq_weight, dk_weight, stream)


def kda_paged_append_fp8(k, v, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, cu_seqlens, T,
                         B, Hkv, D, pages, page_size, max_pages, k_stride, v_stride, k_page_stride,
                         k_token_stride, k_head_stride, v_page_stride, v_token_stride, v_head_stride,
                         k_scale_stride, v_scale_stride, stream) -> int:
    """The C entry point that fills an 8-bit cache, pointers as ints (0 = NULL)."""
    return lib().kda_paged_append_fp8(k, v, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens,
                                      cu_seqlens, T, B, Hkv, D, pages, page_size, max_pages, k_stride,
                                      v_stride, k_page_stride, k_token_stride, k_head_stride,
                                      v_page_stride, v_token_stride, v_head_stride, k_scale_stride,
                                      v_scale_stride, stream)


def kda_paged_decode_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, B, Hq, Hkv, D,
                         pages, page_size, max_pages, k_page_stride, k_token_stride, k_head_stride,
                         v_page_stride, v_token_stride, v_head_stride, k_scale_stride, v_scale_stride,
                         scale, out, lse, stream) -> int:
    """The C entry point of the attention over an 8-bit cache, pointers as ints (0 = NULL)."""
    return lib().kda_paged_decode_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, B, Hq,
                                      Hkv, D, pages, page_size, max_pages, k_page_stride, k_token_stride,
                                      k_head_stride, v_page_stride, v_token_stride, v_head_stride,
                                      k_scale_stride, v_scale_stride, scale, out, lse, stream)


def kda_status_string(code: int) -> str:
    return lib().kda_status_string(int(code)).decode()


def kda_last_device_error(stream=0) -> int:
    return lib().kda_last_device_error(stream)


def kda_workspace_release() -> int:
    return lib().kda_workspace_release()


def kda_workspace_bytes(B, T, H, N, has_cu_seqlens) -> int:
    return lib().kda_workspace_bytes(B, T, H, N, int(bool(has_cu_seqlens)))


def kda_stage_timing_begin(max_calls: int) -> int:
    return lib().kda_stage_timing_begin(int(max_calls))


def kda_stage_timing_end():
    """Returns (status, intra_ms_mean, recurrent_ms_mean, calls)."""
    a, b, n = ctypes.c_double(), ctypes.c_double(), ctypes.c_int()
    rc = lib().kda_stage_timing_end(ctypes.byref(a), ctypes.byref(b), ctypes.byref(n))
    return rc, a.value, b.value, n.value


def kda_set_recurrent_impl(impl: int) -> int:
    """1 = 16-token chunks (default), 3 = 64-token chunks on tcgen05 (two
    kernels), 4 = 64-token chunks in one cooperative launch."""
    return lib().kda_set_recurrent_impl(int(impl))


def kda_set_scan_segments(segments: int) -> int:
    """Segment-parallel scan for fixed-length calls: 0 = automatic, 1 = off,
    P >= 2 = P segments per sequence."""
    return lib().kda_set_scan_segments(int(segments))


def kda_set_backward_impl(impl: int) -> int:
    """Gradients: 0 = chunked (default), 1 = token-serial."""
    return lib().kda_set_backward_impl(int(impl))


def kda_test_stall_recurrent(chunk: int, wait_ns: int = 0) -> int:
    """Test hook: the recurrent kernel's record producer stops before `chunk`
    and its waits give up after `wait_ns` (-1: off)."""
    return lib().kda_test_stall_recurrent(int(chunk), int(wait_ns))


def kda_test_stall_scan(chunk: int) -> int:
    """Test hook: the state space scan's blocks copy the tiles of their first `chunk`
    chunks only, and their waits run out (-1: off)."""
    return lib().kda_test_stall_scan(int(chunk))


def kda_test_stall_qk_norm_rope(batch: int) -> int:
    """Test hook: the warps of the norms with the rotation and of their gradients ask for no more
    heads once they have taken `batch` batches, and their waits run out (-1: off)."""
    return lib().kda_test_stall_qk_norm_rope(int(batch))


def kda_test_stall_paged_fp8(tile: int) -> int:
    """Test hook: the blocks of the attention over an 8-bit cache copy their first `tile` tiles
    only, and their waits run out (-1: off)."""
    return lib().kda_test_stall_paged_fp8(int(tile))


def kda_test_conv_backward_plan(x, d_out, dx, tokens, D, W, x_stride, dout_stride, dx_stride,
                                flags):
    """Test hook: (status, (scratch bytes, channels of a block, blocks along the
    channels, tokens of a run, tiles)) of the convolution's gradient."""
    plan = (ctypes.c_int64 * 5)()
    rc = lib().kda_test_conv_backward_plan(x, d_out, dx, tokens, D, W, x_stride, dout_stride,
                                           dx_stride, flags, plan)
    return rc, tuple(plan)


def kda_build_info() -> str:
    return lib().kda_build_info().decode()


# ------------------------------------------------------------ torch front

def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _flags(normalize_qk, gate_logits):
    return (PRE_NORM_QK if normalize_qk else 0) | (PRE_GATE_LOGITS if gate_logits else 0)


def chunk_prefill(q, k, v, g, beta, initial_state=None, cu_seqlens=None, scale=None, out=None,
                  final_state=None, output_final_state=True, stream=None, normalize_qk=False,
                  gate_logits=False):
    """Chunked KDA prefill on the current CUDA device.

    q, k, v: bf16 [T, H, 128] (packed or one sequence) or [B, T, H, 128];
    g: fp32 like q; beta: fp32 [..., H]; initial_state: fp32 [N, H, 128, 128]
    or None; cu_seqlens: int32 [N+1] on the device or None. Returns
    (o, final_state) with o bf16 like v and final_state fp32 [N, H, 128, 128]
    (None if output_final_state is False and final_state is None).
    normalize_qk / gate_logits: q, k are raw projections to be L2-normalised,
    and g holds gate logits whose logsigmoid is the log decay (done in the
    kernels).
    """
    import torch

    if q.dim() == 4:
        B, T, H, K = q.shape
    elif q.dim() == 3:
        B, (T, H, K) = 1, q.shape
    else:
        raise ValueError("q must be [T, H, K] or [B, T, H, K]")
    V = v.shape[-1]
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError("cu_seqlens needs B == 1")
        if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
            raise ValueError("cu_seqlens must be an int32 CUDA tensor")
        N = cu_seqlens.numel() - 1
    else:
        N = B
    for name, t, dt in (("q", q, torch.bfloat16), ("k", k, torch.bfloat16),
                        ("v", v, torch.bfloat16), ("g", g, torch.float32),
                        ("beta", beta, torch.float32)):
        if t.dtype != dt:
            raise ValueError(f"{name} must be {dt}")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if k.shape != q.shape or g.shape != q.shape or v.shape[:-1] != q.shape[:-1]:
        raise ValueError("q, k, g must share a shape and v must match it but for the last dim")
    if tuple(beta.shape) != tuple(q.shape[:-1]):
        raise ValueError("beta must be q.shape[:-1]")
    if initial_state is not None:
        if initial_state.dtype != torch.float32 or not initial_state.is_contiguous():
            raise ValueError("initial_state must be a contiguous fp32 tensor")
        if tuple(initial_state.shape) != (N, H, K, V):
            raise ValueError(f"initial_state must be [{N}, {H}, {K}, {V}]")
    if scale is None:
        scale = 1.0 / math.sqrt(K)
    if out is None:
        out = torch.empty_like(v)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, K, V), dtype=torch.float32, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    flags = _flags(normalize_qk, gate_logits)
    if flags:
        rc = kda_chunk_prefill_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                  _ptr(initial_state), _ptr(cu_seqlens), B, T, H, K, V, N,
                                  float(scale), flags, _ptr(out), _ptr(final_state), stream)
    else:
        rc = kda_chunk_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                               _ptr(initial_state), _ptr(cu_seqlens), B, T, H, K, V, N,
                               float(scale), _ptr(out), _ptr(final_state), stream)
    if rc != 0:
        raise KdaError(rc, "kda_chunk_prefill")
    return out, final_state


def decode_step(q, k, v, g, beta, state=None, scale=None, out=None, state_out=None,
                in_place=False, stream=None, normalize_qk=False, gate_logits=False):
    """One decode token per sequence on the current CUDA device.

    q, k, v: bf16 [N, H, 128]; g: fp32 [N, H, 128]; beta: fp32 [N, H];
    state: fp32 [N, H, 128, 128] or None (zero state). Returns (o, new_state).
    With in_place=True the new state is written over `state`. normalize_qk /
    gate_logits as for chunk_prefill.
    """
    import torch

    if q.dim() != 3:
        raise ValueError("q must be [N, H, K]")
    N, H, K = q.shape
    V = v.shape[-1]
    for name, t, dt in (("q", q, torch.bfloat16), ("k", k, torch.bfloat16),
                        ("v", v, torch.bfloat16), ("g", g, torch.float32),
                        ("beta", beta, torch.float32)):
        if t.dtype != dt:
            raise ValueError(f"{name} must be {dt}")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if k.shape != q.shape or g.shape != q.shape or v.shape[:-1] != q.shape[:-1]:
        raise ValueError("q, k, g must share a shape and v must match it but for the last dim")
    if tuple(beta.shape) != (N, H):
        raise ValueError("beta must be [N, H]")
    if state is not None:
        if state.dtype != torch.float32 or not state.is_contiguous():
            raise ValueError("state must be a contiguous fp32 tensor")
        if tuple(state.shape) != (N, H, K, V):
            raise ValueError(f"state must be [{N}, {H}, {K}, {V}]")
    if in_place:
        if state is None:
            raise ValueError("in_place needs a state")
        state_out = state
    elif state_out is None:
        state_out = torch.empty((N, H, K, V), dtype=torch.float32, device=q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(K)
    if out is None:
        out = torch.empty_like(v)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    rc = kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
                         _ptr(state_out), N, H, K, V, float(scale),
                         _flags(normalize_qk, gate_logits), _ptr(out), stream)
    if rc != 0:
        raise KdaError(rc, "kda_decode_step")
    return out, state_out


def chunk_prefill_backward(q, k, v, g, beta, d_out, initial_state=None, cu_seqlens=None,
                           scale=None, d_final_state=None, d_initial_state=True, stream=None):
    """Gradients of ``chunk_prefill`` on the current CUDA device.

    Inputs as for chunk_prefill (no preprocessing flags), plus d_out (bf16,
    like v: dL/do) and d_final_state (fp32 [N, H, 128, 128] or None = 0).
    Returns (dq, dk, dv, dg, dbeta, d_initial_state), fp32, shaped like q, k,
    v, g, beta and [N, H, 128, 128]; d_initial_state is None when asked for
    with False.
    """
    import torch

    if q.dim() == 4:
        B, T, H, K = q.shape
    elif q.dim() == 3:
        B, (T, H, K) = 1, q.shape
    else:
        raise ValueError("q must be [T, H, K] or [B, T, H, K]")
    V = v.shape[-1]
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError("cu_seqlens needs B == 1")
        if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
            raise ValueError("cu_seqlens must be an int32 CUDA tensor")
        N = cu_seqlens.numel() - 1
    else:
        N = B
    for name, t, dt in (("q", q, torch.bfloat16), ("k", k, torch.bfloat16),
                        ("v", v, torch.bfloat16), ("g", g, torch.float32),
                        ("beta", beta, torch.float32), ("d_out", d_out, torch.bfloat16)):
        if t.dtype != dt:
            raise ValueError(f"{name} must be {dt}")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if k.shape != q.shape or g.shape != q.shape or v.shape[:-1] != q.shape[:-1]:
        raise ValueError("q, k, g must share a shape and v must match it but for the last dim")
    if d_out.shape != v.shape:
        raise ValueError("d_out must be shaped like v")
    if tuple(beta.shape) != tuple(q.shape[:-1]):
        raise ValueError("beta must be q.shape[:-1]")
    for name, t in (("initial_state", initial_state), ("d_final_state", d_final_state)):
        if t is not None:
            if t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda:
                raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor")
            if tuple(t.shape) != (N, H, K, V):
                raise ValueError(f"{name} must be [{N}, {H}, {K}, {V}]")
    if scale is None:
        scale = 1.0 / math.sqrt(K)
    f32 = dict(dtype=torch.float32, device=q.device)
    dq, dk, dg = (torch.empty(q.shape, **f32) for _ in range(3))
    dv = torch.empty(v.shape, **f32)
    dbeta = torch.empty(beta.shape, **f32)
    ds0 = torch.empty((N, H, K, V), **f32) if d_initial_state else None
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    rc = kda_chunk_prefill_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                    _ptr(initial_state), _ptr(cu_seqlens), B, T, H, K, V, N,
                                    float(scale), _ptr(d_out), _ptr(d_final_state), _ptr(dq),
                                    _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(ds0), stream)
    if rc != 0:
        raise KdaError(rc, "kda_chunk_prefill_backward")
    return dq, dk, dv, dg, dbeta, ds0


def _batch(t, rows_dims, cu_seqlens, name):
    """(B, T, N) of a [T, ...] or [B, T, ...] tensor whose rows have rows_dims dims."""
    import torch

    if t.dim() == rows_dims + 2:
        B, T = t.shape[:2]
    elif t.dim() == rows_dims + 1:
        B, T = 1, t.shape[0]
    else:
        raise ValueError(f"{name} must be [T, ...] or [B, T, ...]")
    if cu_seqlens is None:
        return B, T, B
    if B != 1:
        raise ValueError("cu_seqlens needs B == 1")
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous int32 CUDA tensor")
    return B, T, cu_seqlens.numel() - 1


def _row_stride(t, rows_dims, name):
    """Elements between the rows of a [T, ...] or [B, T, ...] tensor: rows are
    contiguous inside, evenly spaced, and batches follow one another."""
    shape = t.shape
    if rows_dims == 1:
        expect = shape[-1]
    elif rows_dims == 2:
        expect = shape[-1] * shape[-2]
    else:
        expect = math.prod(shape[-rows_dims:])
    if t.is_contiguous():
        return expect
    strides = t.stride()
    if len(shape) == 3 and rows_dims == 2 and strides[2] == 1 and strides[1] == shape[2]:
        if strides[0] >= expect:
            return strides[0]   # (the usual slice of a projection)
    inner = 1
    for i in range(1, rows_dims + 1):
        if strides[-i] != inner and shape[-i] > 1:
            raise ValueError(f"{name} must be contiguous within a token")
        inner *= shape[-i]
    at = len(shape) - rows_dims - 1
    stride = strides[at] if shape[at] > 1 else expect
    if at == 1 and shape[0] > 1:
        if shape[1] == 1:
            stride = strides[0]
        elif strides[0] != shape[1] * stride:
            raise ValueError(f"{name}: batches must follow one another at the token stride")
    if stride < expect:
        raise ValueError(f"{name}: tokens must not overlap")
    return stride


def _need(name, t, dtype, shape, contiguous=True):
    if (t.dtype is dtype and t.shape == shape and t.is_cuda
            and (not contiguous or t.is_contiguous())):
        return
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}")
    raise ValueError(f"{name} must be a {'contiguous ' if contiguous else ''}CUDA tensor")


def _need_rows(name, t, dtype, shape, dims=2):
    """_need for rows of `dims` dimensions that may be strided; returns their stride."""
    if not (t.dtype is dtype and t.shape == shape and t.is_cuda):
        _need(name, t, dtype, shape, contiguous=False)
    if dims == 2 and len(shape) == 3:
        row, head, channel = t.stride()
        if channel == 1 and head == shape[2] and row >= shape[1] * head and shape[0] > 1:
            return row
    return _row_stride(t, dims, name)


def _conv_flags(activation):
    if activation not in (None, "silu"):
        raise ValueError("activation must be None or 'silu'")
    return CONV_SILU if activation == "silu" else 0


def _filter(x, weight, bias):
    import torch

    if weight.dim() != 2:
        raise ValueError("weight must be [D, W]")
    D, W = weight.shape
    if x.dtype != torch.bfloat16 or not x.is_cuda:
        raise ValueError("x must be a bfloat16 CUDA tensor")
    if x.shape[-1] != D:
        raise ValueError("x must have weight.shape[0] channels")
    _need("weight", weight, torch.float32, (D, W))
    if bias is not None:
        _need("bias", bias, torch.float32, (D,))
    return D, W


def _current_stream(t, stream):
    import torch

    # the raw handle: torch.cuda.current_stream() builds a Stream object first
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else stream


def short_conv(x, weight, bias=None, initial_state=None, cu_seqlens=None, activation="silu",
               out=None, final_state=None, output_final_state=True, stream=None):
    """Short causal convolution on the current CUDA device, one filter per channel.

    x: bf16 [T, D] (packed or one sequence) or [B, T, D], tokens any even
    stride apart (a slice of a fused projection); weight: fp32 [D, W], W = 2..4
    (weight[:, W-1] meets the token itself); bias: fp32 [D] or None;
    initial_state: bf16 [N, W-1, D], the rows before each sequence, newest
    last, or None; cu_seqlens: int32 [N+1] on the device or None; activation:
    "silu" or None. Returns (out, final_state): bf16 like x and the last W-1
    rows [N, W-1, D] (None if output_final_state is False and final_state is
    None).
    """
    import torch

    flags = _conv_flags(activation)
    D, W = _filter(x, weight, bias)
    B, T, N = _batch(x, 1, cu_seqlens, "x")
    if initial_state is not None:
        _need("initial_state", initial_state, torch.bfloat16, (N, W - 1, D))
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _need("out", out, torch.bfloat16, x.shape, contiguous=False)
    if final_state is not None:
        _need("final_state", final_state, torch.bfloat16, (N, W - 1, D))
    elif output_final_state:
        final_state = torch.empty((N, W - 1, D), dtype=torch.bfloat16, device=x.device)
    rc = lib().kda_short_conv(_ptr(x), _ptr(weight), _ptr(bias), _ptr(initial_state), _ptr(cu_seqlens),
                        B, T, D, W, N, _row_stride(x, 1, "x"), flags, _ptr(out),
                        _row_stride(out, 1, "out"), _ptr(final_state), _current_stream(x, stream))
    if rc != 0:
        raise KdaError(rc, "kda_short_conv")
    return out, final_state


def short_conv_step(x, weight, state=None, bias=None, activation="silu", out=None, state_out=None,
                    in_place=False, stream=None):
    """The convolution for one new token per sequence on the current CUDA device.

    x: bf16 [N, D]; state: bf16 [N, W-1, D], the last rows, newest last, or
    None (zeros); the rest as for short_conv. Returns (out, new_state). With
    in_place=True the new state is written over `state`.
    """
    import torch

    flags = _conv_flags(activation)
    if x.dim() != 2:
        raise ValueError("x must be [N, D]")
    D, W = _filter(x, weight, bias)
    N = x.shape[0]
    if state is not None:
        _need("state", state, torch.bfloat16, (N, W - 1, D))
    if in_place:
        if state is None:
            raise ValueError("in_place needs a state")
        state_out = state
    elif state_out is None:
        state_out = torch.empty((N, W - 1, D), dtype=torch.bfloat16, device=x.device)
    else:
        _need("state_out", state_out, torch.bfloat16, (N, W - 1, D))
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _need("out", out, torch.bfloat16, x.shape, contiguous=False)
    rc = lib().kda_short_conv_step(_ptr(x), _ptr(weight), _ptr(bias), _ptr(state), N, D, W,
                             _row_stride(x, 1, "x"), flags, _ptr(out), _row_stride(out, 1, "out"),
                             _ptr(state_out), _current_stream(x, stream))
    if rc != 0:
        raise KdaError(rc, "kda_short_conv_step")
    return out, state_out


def short_conv_backward(x, weight, d_out, bias=None, initial_state=None, cu_seqlens=None,
                        activation="silu", d_final_state=None, d_initial_state=True, dx=None,
                        stream=None):
    """Gradients of ``short_conv`` on the current CUDA device.

    Inputs as for short_conv, plus d_out (bf16 or fp32, shaped like x) and
    d_final_state (fp32 [N, W-1, D] or None = 0). Returns (dx, dweight, dbias,
    d_initial_state): bf16 like x (written to `dx` if given, which may be
    strided), fp32 [D, W], fp32 [D] (None without a bias) and fp32
    [N, W-1, D] (None when asked for with False).
    """
    import torch

    flags = _conv_flags(activation)
    D, W = _filter(x, weight, bias)
    B, T, N = _batch(x, 1, cu_seqlens, "x")
    if d_out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("d_out must be bfloat16 or float32")
    _need("d_out", d_out, d_out.dtype, x.shape, contiguous=False)
    if d_out.dtype == torch.float32:
        flags |= CONV_DOUT_FP32
    if initial_state is not None:
        _need("initial_state", initial_state, torch.bfloat16, (N, W - 1, D))
    if d_final_state is not None:
        _need("d_final_state", d_final_state, torch.float32, (N, W - 1, D))
    if dx is None:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _need("dx", dx, torch.bfloat16, x.shape, contiguous=False)
    f32 = dict(dtype=torch.float32, device=x.device)
    dweight = torch.empty((D, W), **f32)
    dbias = torch.empty((D,), **f32) if bias is not None else None
    dh = torch.empty((N, W - 1, D), **f32) if d_initial_state else None
    rc = lib().kda_short_conv_backward(
        _ptr(x), _ptr(weight), _ptr(bias), _ptr(initial_state), _ptr(cu_seqlens), B, T, D, W, N,
        _row_stride(x, 1, "x"), flags, _ptr(d_out), _row_stride(d_out, 1, "d_out"),
        _ptr(d_final_state), _ptr(dx), _row_stride(dx, 1, "dx"), _ptr(dweight), _ptr(dbias),
        _ptr(dh), _current_stream(x, stream))
    if rc != 0:
        raise KdaError(rc, "kda_short_conv_backward")
    return dx, dweight, dbias, dh


def _ssm_inputs(x, dt, a, b, c, d, dt_bias, rows):
    """Checks the scan's inputs; returns (H, P, G, n)."""
    import torch

    H, P = x.shape[-2:]
    G, n = b.shape[-2:]
    _need("x", x, torch.bfloat16, (*rows, H, P), contiguous=False)
    _need("dt", dt, torch.float32, (*rows, H), contiguous=False)
    _need("b", b, torch.bfloat16, (*rows, G, n), contiguous=False)
    _need("c", c, torch.bfloat16, (*rows, G, n), contiguous=False)
    for name, t in (("a", a), ("d", d), ("dt_bias", dt_bias)):
        if t is not None or name == "a":
            _need(name, t, torch.float32, (H,))
    if G == 0 or H % G:
        raise ValueError("the heads must be a multiple of the groups of b and c")
    return H, P, G, n


def ssm_prefill(x, dt, a, b, c, d=None, dt_bias=None, initial_state=None, cu_seqlens=None,
                dt_softplus=False, out=None, final_state=None, output_final_state=True,
                stream=None):
    """Selective state space scan over a batch of sequences on the current CUDA device.

    S_t = exp(a delta_t) S_{t-1} + delta_t b_t x_t^T, y_t = S_t^T c_t + d x_t, with
    delta = dt + dt_bias, through softplus if dt_softplus.
    x: bf16 [T, H, P] (packed or one sequence) or [B, T, H, P]; dt: fp32
    [..., H]; b, c: bf16 [..., G, n], shared by H/G heads each; tokens of x, dt,
    b and c any even stride apart (slices of a fused projection); a: fp32 [H]
    (negative); d, dt_bias: fp32 [H] or None; initial_state: fp32 [N, H, n, P]
    or None; cu_seqlens: int32 [N+1] on the device or None. P and n are 64 or
    128. Returns (out, final_state): bf16 like x (contiguous), fp32
    [N, H, n, P] (None if output_final_state is False and final_state is None).
    """
    import torch

    B, T, N = _batch(x, 2, cu_seqlens, "x")
    H, P, G, n = _ssm_inputs(x, dt, a, b, c, d, dt_bias, x.shape[:-2])
    if initial_state is not None:
        _need("initial_state", initial_state, torch.float32, (N, H, n, P))
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _need("out", out, torch.bfloat16, x.shape)
    if final_state is not None:
        _need("final_state", final_state, torch.float32, (N, H, n, P))
    elif output_final_state:
        final_state = torch.empty((N, H, n, P), dtype=torch.float32, device=x.device)
    rc = lib().kda_ssm_prefill(
        _ptr(x), _ptr(dt), _ptr(a), _ptr(b), _ptr(c), _ptr(d), _ptr(dt_bias),
        _ptr(initial_state), _ptr(cu_seqlens), B, T, H, P, G, n, N, _row_stride(x, 2, "x"),
        _row_stride(dt, 1, "dt"), _row_stride(b, 2, "b"), _row_stride(c, 2, "c"),
        SSM_DT_SOFTPLUS if dt_softplus else 0, _ptr(out), _ptr(final_state),
        _current_stream(x, stream))
    if rc != 0:
        raise KdaError(rc, "kda_ssm_prefill")
    return out, final_state


def ssm_step(x, dt, a, b, c, state=None, d=None, dt_bias=None, dt_softplus=False, out=None,
             state_out=None, in_place=False, stream=None):
    """The scan for one new token per sequence on the current CUDA device.

    x: bf16 [N, H, P]; dt: fp32 [N, H]; b, c: bf16 [N, G, n]; state: fp32
    [N, H, n, P] or None (zeros); the rest as for ssm_prefill. Returns
    (out, new_state). With in_place=True the new state is written over `state`.
    """
    import torch

    if x.dim() != 3:
        raise ValueError("x must be [N, H, P]")
    N = x.shape[0]
    H, P, G, n = _ssm_inputs(x, dt, a, b, c, d, dt_bias, (N,))
    if state is not None:
        _need("state", state, torch.float32, (N, H, n, P))
    if in_place:
        if state is None:
            raise ValueError("in_place needs a state")
        state_out = state
    elif state_out is None:
        state_out = torch.empty((N, H, n, P), dtype=torch.float32, device=x.device)
    else:
        _need("state_out", state_out, torch.float32, (N, H, n, P))
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _need("out", out, torch.bfloat16, x.shape)
    rc = lib().kda_ssm_step(_ptr(x), _ptr(dt), _ptr(a), _ptr(b), _ptr(c), _ptr(d), _ptr(dt_bias),
                      _ptr(state), N, H, P, G, n, _row_stride(x, 2, "x"),
                      _row_stride(dt, 1, "dt"), _row_stride(b, 2, "b"), _row_stride(c, 2, "c"),
                      SSM_DT_SOFTPLUS if dt_softplus else 0, _ptr(out), _ptr(state_out),
                      _current_stream(x, stream))
    if rc != 0:
        raise KdaError(rc, "kda_ssm_step")
    return out, state_out


def paged_decode(q, k_cache, v_cache, page_table, seq_lens, scale=None, out=None, lse=None,
                 stream=None):
    """Attention of one new token per sequence over a paged cache, current CUDA device.

    q: bf16 [B, Hq, D], D = 64 or 128; k_cache, v_cache: bf16
    [pages, page_size, Hkv, D], contiguous inside a page (both may be views of
    one cache); page_table: int32 [B, max_pages]; seq_lens: int32 [B], the new
    token included (0: out = 0, lse = -inf); scale: 1/sqrt(D) by default.
    Returns (out, lse): bf16 like q and fp32 [B, Hq] (natural logarithm).
    """
    import torch

    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [B, Hq, D] and the caches [pages, page_size, Hkv, D]")
    B, Hq, D = q.shape
    pages, page_size, Hkv, _ = k_cache.shape
    _need("q", q, torch.bfloat16, (B, Hq, D))
    _need("k_cache", k_cache, torch.bfloat16, (pages, page_size, Hkv, D), contiguous=False)
    _need("v_cache", v_cache, torch.bfloat16, (pages, page_size, Hkv, D), contiguous=False)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    _need("page_table", page_table, torch.int32, (B, page_table.shape[1]))
    _need("seq_lens", seq_lens, torch.int32, (B,))
    if scale is None:
        scale = 1.0 / math.sqrt(max(D, 1))   # (D = 0 is refused below)
    if out is None:
        out = torch.empty_like(q)
    else:
        _need("out", out, torch.bfloat16, q.shape)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    else:
        _need("lse", lse, torch.float32, (B, Hq))
    rc = lib().kda_paged_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(seq_lens),
                          B, Hq, Hkv, D, pages, page_size, page_table.shape[1],
                          _row_stride(k_cache, 3, "k_cache"), _row_stride(v_cache, 3, "v_cache"),
                          float(scale), _ptr(out), _ptr(lse), _current_stream(q, stream))
    if rc != 0:
        raise KdaError(rc, "kda_paged_decode")
    return out, lse


def page_plan(page_table, seq_lens, new_lens, free_pages, free_count, page_size, tokens, release=None,
              in_place=False, stream=None):
    """Page tables, positions and slots of a batch's next tokens, on the current CUDA device.

    page_table: int32 [B, max_pages]; seq_lens: int32 [B], the tokens each slot holds;
    new_lens: int32 [B], those that join; free_pages: int32 [pool], a stack of the
    pages that nobody holds, the first free_count (int32 [1]) of them; release: bool
    or uint8 [B] or None, slots whose pages are given back first; tokens: rows of the
    positions and slots, at least the new tokens. Returns (page_table, seq_lens,
    free_pages, free_count, cu_seqlens, positions, slots): the first four after the
    call (with in_place=True the tensors given, updated), int32 [B + 1], int32
    [tokens] and int64 [tokens]. Rows behind the last new token have position 0 and
    slot -1. Too few pages and bad lengths are reported by check_device_error(), and
    nothing is planned then.
    """
    import torch

    if page_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("page_table must be [B, max_pages] and free_pages [pool]")
    B, width = page_table.shape
    given = (page_table, seq_lens, free_pages, free_count)
    _need("page_table", page_table, torch.int32, (B, width))
    _need("seq_lens", seq_lens, torch.int32, (B,))
    _need("new_lens", new_lens, torch.int32, (B,))
    _need("free_pages", free_pages, torch.int32, free_pages.shape)
    _need("free_count", free_count, torch.int32, (1,))
    if release is not None:
        if release.dtype not in (torch.bool, torch.uint8):
            raise ValueError("release must be bool or uint8")
        _need("release", release, release.dtype, (B,))
    tokens, device = int(tokens), page_table.device
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    after = given if in_place else tuple(torch.empty_like(t) for t in given)
    cu = torch.empty((B + 1,), dtype=torch.int32, device=device)
    positions = torch.empty((tokens,), dtype=torch.int32, device=device)
    slots = torch.empty((tokens,), dtype=torch.int64, device=device)
    rc = lib().kda_page_plan(_ptr(page_table), _ptr(seq_lens), _ptr(new_lens), _ptr(release),
                             _ptr(free_pages), _ptr(free_count), B, width, free_pages.shape[0],
                             page_size, tokens, _ptr(after[0]), _ptr(after[1]), _ptr(after[2]),
                             _ptr(after[3]), _ptr(cu), _ptr(positions), _ptr(slots),
                             _current_stream(page_table, stream))
    if rc != 0:
        raise KdaError(rc, "kda_page_plan")
    return (*after, cu, positions, slots)


def _heads_inputs(q, k, q_weight, k_weight, inv_freq, positions):
    """Checks of the norms' inputs; returns (T, Hq, Hk, D, R, q's and k's stride)."""
    import torch

    shape, bf16 = q.shape, torch.bfloat16
    if len(shape) == 3:
        T, Hq, D = shape
    elif len(shape) == 4:
        T, Hq, D = shape[0] * shape[1], shape[2], shape[3]
    else:
        raise ValueError("q must be [T, Hq, D] or [B, T, Hq, D]")
    q_stride = _need_rows("q", q, bf16, shape)
    Hk = k_stride = R = 0
    if k is not None:
        like = k.shape
        Hk = like[-2] if len(like) == len(shape) else -1
        k_stride = _need_rows("k", k, bf16, (*shape[:-2], Hk, D))
    if q_weight is not None:
        _need("q_weight", q_weight, torch.float32, (D,))
    if k_weight is not None:
        _need("k_weight", k_weight, torch.float32, (D,))
    if inv_freq is not None:
        R = 2 * inv_freq.numel()
        _need("inv_freq", inv_freq, torch.float32, (R // 2,))
        if positions is None:
            raise ValueError("inv_freq needs positions")
        _need("positions", positions, torch.int32, shape[:-2])
    return T, Hq, Hk, D, R, q_stride, k_stride


def _like(name, t, x):
    """An output shaped like x, strided as it likes: given, or made; and its stride."""
    import torch

    if t is not None:
        return t, _need_rows(name, t, torch.bfloat16, x.shape)
    t = torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    return t, t.shape[-1] * t.shape[-2]


def qk_norm_rope(q, k=None, q_weight=None, k_weight=None, inv_freq=None, positions=None, eps=1e-6,
                 interleaved=False, q_out=None, k_out=None, stream=None):
    """Norm of every query and key head and the rotation by its position, current CUDA device.

    x / sqrt(mean(x^2) + eps) * weight over the channels of a head, then the first R
    channels turned by positions * inv_freq, in pairs (i, i + R/2) or, interleaved,
    (2i, 2i + 1). q, k: bf16 [T, H, D] or [B, T, H, D], D = 64, 128 or 256, tokens any
    even stride apart (slices of a fused projection), k may be None; weights: fp32 [D]
    or None; inv_freq: fp32 [R/2] (R a multiple of 16) with positions int32 [T] or
    [B, T], or None (no rotation). q_out and k_out may be q and k (in place). Returns
    (q_out, k_out), bf16 (None without k).
    """
    import torch

    T, Hq, Hk, D, R, q_stride, k_stride = _heads_inputs(q, k, q_weight, k_weight, inv_freq, positions)
    q_out, qo_stride = _like("q_out", q_out, q)
    k_out, ko_stride = _like("k_out", k_out, k) if k is not None else (None, 0)
    rc = lib().kda_qk_norm_rope(
        q.data_ptr(), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(inv_freq), _ptr(positions), T, Hq, Hk,
        D, R, q_stride, k_stride, eps, ROPE_INTERLEAVED if interleaved else 0, q_out.data_ptr(), qo_stride,
        _ptr(k_out), ko_stride, _current_stream(q, stream))
    if rc != 0:
        raise KdaError(rc, "kda_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(q, k, dq_out, dk_out, q_weight=None, k_weight=None, inv_freq=None,
                          positions=None, eps=1e-6, interleaved=False, dq=None, dk=None, stream=None):
    """Gradients of ``qk_norm_rope`` on the current CUDA device.

    Inputs as there (q and k as given to it), plus dq_out and dk_out, bf16 or both fp32,
    shaped like q and k. Returns (dq, dk, dq_weight, dk_weight): bf16 like q and k
    (written to `dq` and `dk` if given, which may be strided), fp32 [D] (None for
    weights that are None; dk and dk_weight None without k).
    """
    import torch

    T, Hq, Hk, D, R, q_stride, k_stride = _heads_inputs(q, k, q_weight, k_weight, inv_freq, positions)
    flags, dtype = ROPE_INTERLEAVED if interleaved else 0, dq_out.dtype
    if dtype is torch.float32:
        flags |= ROPE_DOUT_FP32
    elif dtype is not torch.bfloat16:
        raise ValueError("dq_out must be bfloat16 or float32")
    dqo_stride = _need_rows("dq_out", dq_out, dtype, q.shape)
    dko_stride = dk_stride = 0
    if k is not None:
        if dk_out is None:
            raise ValueError("dk_out is missing")
        dko_stride = _need_rows("dk_out", dk_out, dtype, k.shape)
        dk, dk_stride = _like("dk", dk, k)
    elif dk_out is not None:
        raise ValueError("dk_out needs k")
    else:
        dk = None
    dq, dq_stride = _like("dq", dq, q)
    dqw = torch.empty_like(q_weight) if q_weight is not None else None
    dkw = torch.empty_like(k_weight) if k_weight is not None and k is not None else None
    rc = lib().kda_qk_norm_rope_backward(
        q.data_ptr(), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(inv_freq), _ptr(positions), T, Hq, Hk,
        D, R, q_stride, k_stride, eps, flags, dq_out.data_ptr(), dqo_stride, _ptr(dk_out), dko_stride,
        dq.data_ptr(), dq_stride, _ptr(dk), dk_stride, _ptr(dqw), _ptr(dkw), _current_stream(q, stream))
    if rc != 0:
        raise KdaError(rc, "kda_qk_norm_rope_backward")
    return dq, dk, dqw, dkw


def _fp8_cache(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, B):
    """Checks of an 8-bit cache; returns (pages, page_size, Hkv, D, max_pages, strides)."""
    import torch

    shape, table = k_cache.shape, page_table.shape
    if len(shape) != 4:
        raise ValueError("the caches must be [pages, page_size, Hkv, D]")
    if len(table) != 2:
        raise ValueError("page_table must be [B, max_pages]")
    f8, width = torch.float8_e4m3fn, table[1]
    pages, page_size, Hkv, D = shape
    _need("k_cache", k_cache, f8, shape, contiguous=False)
    _need("v_cache", v_cache, f8, shape, contiguous=False)
    *k_strides, k_channel = k_cache.stride()
    *v_strides, v_channel = v_cache.stride()
    if (k_channel != 1 or v_channel != 1) and D > 1:
        raise ValueError(f"{'v' if k_channel == 1 else 'k'}_cache must be contiguous within a head")
    strides = (*k_strides, *v_strides, _need_rows("k_scale", k_scale, torch.float32, (pages, Hkv), 1),
               _need_rows("v_scale", v_scale, torch.float32, (pages, Hkv), 1))
    _need("page_table", page_table, torch.int32, (B, width))
    _need("seq_lens", seq_lens, torch.int32, (B,))
    return pages, page_size, Hkv, D, width, strides


def paged_append_fp8(k, v, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, cu_seqlens=None,
                     stream=None):
    """New keys and values into a paged 8-bit cache, on the current CUDA device.

    k, v: bf16 [T, Hkv, D], D = 64 or 128, tokens any even stride apart; k_cache, v_cache:
    float8_e4m3fn [pages, page_size, Hkv, D] with channels contiguous and any other strides;
    k_scale, v_scale: fp32 [pages, Hkv], powers of two that this call settles (a page's scale
    only grows while it is filled); page_table: int32 [B, max_pages]; seq_lens: int32 [B], the
    new tokens included; cu_seqlens: int32 [B + 1], the rows of each slot, which go to its last
    positions, or None (T = B, one token each). Writes the caches and scales in place.
    """
    import torch

    if k.dim() != 3:
        raise ValueError("k must be [T, Hkv, D]")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    T, B = k.shape[0], page_table.shape[0]
    pages, page_size, Hkv, D, width, strides = _fp8_cache(k_cache, v_cache, k_scale, v_scale, page_table,
                                                          seq_lens, B)
    rows = (T, Hkv, D)
    k_stride = _need_rows("k", k, torch.bfloat16, rows)
    v_stride = _need_rows("v", v, torch.bfloat16, rows)
    if cu_seqlens is None:
        if T != B:
            raise ValueError("without cu_seqlens there is one row per slot")
    else:
        _need("cu_seqlens", cu_seqlens, torch.int32, (B + 1,))
    rc = lib().kda_paged_append_fp8(
        k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), _ptr(cu_seqlens), T, B, Hkv, D,
        pages, page_size, width, k_stride, v_stride, *strides, _current_stream(k, stream))
    if rc != 0:
        raise KdaError(rc, "kda_paged_append_fp8")


def paged_decode_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, scale=None, out=None,
                     lse=None, stream=None):
    """Attention of one new token per sequence over a paged 8-bit cache, current CUDA device.

    q: bf16 [B, Hq, D], D = 64 or 128; the cache, its scales, page_table and seq_lens (the new
    token included; 0: out = 0, lse = -inf) as for paged_append_fp8; scale: 1/sqrt(D) by
    default. Returns (out, lse): bf16 like q and fp32 [B, Hq] (natural logarithm).
    """
    import torch

    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q must be [B, Hq, D]")
    B, Hq, D = shape
    pages, page_size, Hkv, dim, width, strides = _fp8_cache(k_cache, v_cache, k_scale, v_scale,
                                                            page_table, seq_lens, B)
    _need("q", q, torch.bfloat16, (B, Hq, dim))
    if scale is None:
        scale = 1.0 / math.sqrt(max(D, 1))   # (D = 0 is refused below)
    if out is None:
        out = torch.empty_like(q)
    else:
        _need("out", out, torch.bfloat16, shape)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    else:
        _need("lse", lse, torch.float32, (B, Hq))
    rc = lib().kda_paged_decode_fp8(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        page_table.data_ptr(), seq_lens.data_ptr(), B, Hq, Hkv, D, pages, page_size, width, *strides,
        scale, out.data_ptr(), lse.data_ptr(), _current_stream(q, stream))
    if rc != 0:
        raise KdaError(rc, "kda_paged_decode_fp8")
    return out, lse


def check_device_error(stream=None):
    """Synchronise the stream and raise if a kernel recorded an error."""
    import torch

    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    rc = kda_last_device_error(stream)
    if rc != 0:
        raise KdaError(rc, "device")
