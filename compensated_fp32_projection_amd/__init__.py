"""Python binding of libcfp32, the compensated-FP32 projection for MI355X.

Argument marshalling only: every step of the projection runs in the HIP
kernels of ``libcfp32.so`` (built by ``compensated_fp32_projection_amd.build``).
PyTorch supplies device memory and the current stream.  There is no CPU
fallback: if the library is missing or the device is not gfx950, calls raise.

Low-level entry points carry the C names and take raw integers (device
pointers, sizes, stream handle):

    cfp32_split, cfp32_gemm, cfp32_gemm_separate_add, cfp32_merge,
    cfp32_linear, cfp32_linear_noalloc, cfp32_linear_workspace_bytes, cfp32_linear_ex,
    cfp32_linear_ex_workspace_bytes, cfp32_linear_geglu,
    cfp32_linear_geglu_workspace_bytes, cfp32_linear_f32, cfp32_qkv_rotary, cfp32_status_string,
    cfp32_last_hip_error, cfp32_attention_prompt, cfp32_attention_decode,
    cfp32_cache_reserve, cfp32_cache_append, cfp32_cache_copy_pages,
    cfp32_cache_fork, cfp32_cache_free, cfp32_cache_compact and the
    *_workspace_bytes of those that take a workspace

Tensor-level helpers (``split``, ``gemm``, ``merge``, ``linear``,
``attention_prompt``, ``attention_decode``, ``cache_*``) check dtype, device
and layout, pass ``data_ptr()`` and the current stream, and raise
``Cfp32Error`` on a non-zero status.  FP16 tensors may be ``torch.float16``
or ``torch.int16``/``torch.uint16`` bit patterns.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcfp32.so")

OK, ERR_INVALID_VALUE, ERR_UNSUPPORTED_DEVICE, ERR_HIP, ERR_TOO_LARGE = 0, 1, 2, 3, 4

EXPORTS = (
    "cfp32_status_string",
    "cfp32_last_hip_error",
    "cfp32_split",
    "cfp32_gemm",
    "cfp32_gemm_separate_add",
    "cfp32_merge",
    "cfp32_linear_workspace_bytes",
    "cfp32_linear",
    "cfp32_linear_noalloc",
    "cfp32_linear_ex_workspace_bytes",
    "cfp32_linear_ex",
    "cfp32_linear_geglu_workspace_bytes",
    "cfp32_linear_geglu",
    "cfp32_linear_f32",
    "cfp32_qkv_rotary",
    "cfp32_attention_prompt_workspace_bytes",
    "cfp32_attention_prompt",
    "cfp32_attention_decode_workspace_bytes",
    "cfp32_attention_decode",
    "cfp32_cache_reserve",
    "cfp32_cache_append",
    "cfp32_cache_copy_pages",
    "cfp32_cache_fork_workspace_bytes",
    "cfp32_cache_fork",
    "cfp32_cache_free",
    "cfp32_cache_compact_workspace_bytes",
    "cfp32_cache_compact",
    "cfp32_rotary_frequencies",
    "cfp32_rotary",
    "cfp32_cache8_append",
    "cfp32_cache8_read",
    "cfp32_cache8_copy_pages",
    "cfp32_cache8_fork",
    "cfp32_cache8_compact",
    "cfp32_attention8_decode_workspace_bytes",
    "cfp32_attention8_decode",
    "cfp32_beam_select_workspace_bytes",
    "cfp32_beam_select",
    "cfp32_beam_reorder",
)

W_KN, W_NK = 0, 1
KV_F32, KV_F16 = 0, 1
CODE_I8, CODE_E4M3 = 0, 1
ROTARY_HALF, ROTARY_INTERLEAVED = 0, 1
ROTARY_PLAIN, ROTARY_LINEAR, ROTARY_NTK, ROTARY_PARTS = 0, 1, 2, 3


class Cache8Desc(ctypes.Structure):
    """cfp32_cache8: the pools of an 8-bit cache as the C calls take them."""

    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v")] + \
        [(n, ctypes.c_int64) for n in ("k_page", "k_head", "k_tok", "v_page", "v_head", "v_tok")] + \
        [(n, ctypes.c_void_p) for n in ("k_scales", "v_scales")] + \
        [(n, ctypes.c_int64) for n in ("ks_page", "ks_head", "vs_page", "vs_head", "P", "Hkv", "page", "block", "D",
                                       "code_type")]


class Cfp32Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = cfp32_status_string(status)
        if status == ERR_HIP:
            msg += f" (hipError_t {cfp32_last_hip_error()})"
        super().__init__(f"{where}: {msg}")


_lib = None


def load_library():
    """Load libcfp32.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m compensated_fp32_projection_amd.build` (no CPU fallback exists)")
    lib = ctypes.CDLL(LIB_PATH)
    # A call that uses a workspace launches several kernels over it, and calls
    # of two threads on one stream may share the helpers' own: they are made
    # with the interpreter's lock held (a few microseconds), as the helpers'
    # native form makes them, so that one's launches do not fall between another's.
    held = ctypes.PyDLL(LIB_PATH)
    for name in ("cfp32_linear", "cfp32_linear_ex", "cfp32_linear_geglu", "cfp32_attention_prompt",
                 "cfp32_attention_decode", "cfp32_cache_fork", "cfp32_cache_compact", "cfp32_cache8_fork",
                 "cfp32_cache8_compact", "cfp32_attention8_decode", "cfp32_beam_select"):
        setattr(lib, name, getattr(held, name))
    P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.cfp32_status_string.argtypes = [I32]
    lib.cfp32_status_string.restype = ctypes.c_char_p
    lib.cfp32_last_hip_error.argtypes = []
    lib.cfp32_last_hip_error.restype = I32
    lib.cfp32_split.argtypes = [P, I64, P, P, I64, I64, I64, P]
    lib.cfp32_split.restype = I32
    lib.cfp32_gemm.argtypes = [P, P, I64, P, I64, P, P, P, I64, I64, I64, I64, P]
    lib.cfp32_gemm.restype = I32
    lib.cfp32_gemm_separate_add.argtypes = [P, P, I64, P, I64, P, P, P, I64, I64, I64, I64, I64, P]
    lib.cfp32_gemm_separate_add.restype = I32
    lib.cfp32_merge.argtypes = [P, P, I64, P, I64, I64, I64, P]
    lib.cfp32_merge.restype = I32
    lib.cfp32_linear_workspace_bytes.argtypes = [I64, I64, I64]
    lib.cfp32_linear_workspace_bytes.restype = ctypes.c_size_t
    lib.cfp32_linear.argtypes = [P, I64, P, I64, P, I64, I64, I64, I64, P, ctypes.c_size_t, P]
    lib.cfp32_linear.restype = I32
    lib.cfp32_linear_noalloc.argtypes = [P, I64, P, I64, P, I64, I64, I64, I64, P]
    lib.cfp32_linear_noalloc.restype = I32
    lib.cfp32_linear_ex_workspace_bytes.argtypes = [I64, I64, I64, I32]
    lib.cfp32_linear_ex_workspace_bytes.restype = ctypes.c_size_t
    lib.cfp32_linear_ex.argtypes = [P, I64, P, I64, I32, P, P, I64, I64, I64, I64, P, ctypes.c_size_t, P]
    lib.cfp32_linear_ex.restype = I32
    lib.cfp32_linear_geglu_workspace_bytes.argtypes = [I64, I64, I64]
    lib.cfp32_linear_geglu_workspace_bytes.restype = ctypes.c_size_t
    lib.cfp32_linear_geglu.argtypes = [P, I64, P, I64, P, P, I64, I64, I64, I64, P, ctypes.c_size_t, P]
    lib.cfp32_linear_geglu.restype = I32
    lib.cfp32_linear_f32.argtypes = [P, I64, P, I64, P, I64, I64, I64, I64, P]
    lib.cfp32_linear_f32.restype = I32
    lib.cfp32_qkv_rotary.argtypes = [P, I64, P, ctypes.c_double, P, P, P, I64, I64, I64, P]
    lib.cfp32_qkv_rotary.restype = I32
    SZ, F64 = ctypes.c_size_t, ctypes.c_double
    view, pool = [P, I64, I64], [P, I64, I64, I64]
    lib.cfp32_attention_prompt_workspace_bytes.argtypes = [I64] * 4 + [I32]
    lib.cfp32_attention_prompt_workspace_bytes.restype = SZ
    lib.cfp32_attention_prompt.argtypes = view * 3 + [I32, P, P] + view + [I64] * 6 + [I32, F64, P, SZ, P]
    lib.cfp32_attention_prompt.restype = I32
    lib.cfp32_attention_decode_workspace_bytes.argtypes = [I64] * 7 + [I32]
    lib.cfp32_attention_decode_workspace_bytes.restype = SZ
    lib.cfp32_attention_decode.argtypes = view + pool * 2 + [I32, I64, I64, P, I64, I64, P, I64] + view + [I64] * 4 + \
        [F64, P, SZ, P]
    lib.cfp32_attention_decode.restype = I32
    lib.cfp32_cache_reserve.argtypes = [P, I64, P, P, P, P, I64, P, P, I64, I64, I64, I64, P]
    lib.cfp32_cache_reserve.restype = I32
    lib.cfp32_cache_append.argtypes = view * 2 + [P] * 3 + pool * 2 + [I32, I64, I64, P] + [I64] * 6 + [P]
    lib.cfp32_cache_append.restype = I32
    lib.cfp32_cache_copy_pages.argtypes = pool * 2 + [I32] + [I64] * 4 + [P, P, I64, P]
    lib.cfp32_cache_copy_pages.restype = I32
    lib.cfp32_cache_fork_workspace_bytes.argtypes = [I64]
    lib.cfp32_cache_fork_workspace_bytes.restype = SZ
    lib.cfp32_cache_fork.argtypes = pool * 2 + [I32] + [I64] * 4 + [P, I64, P, P, P, P, I64, P, P, P] + [I64] * 3 + \
        [P, SZ, P]
    lib.cfp32_cache_fork.restype = I32
    lib.cfp32_cache_free.argtypes = [P, I64, P, P, I64, I64, I64, P]
    lib.cfp32_cache_free.restype = I32
    lib.cfp32_cache_compact_workspace_bytes.argtypes = [I64]
    lib.cfp32_cache_compact_workspace_bytes.restype = SZ
    lib.cfp32_cache_compact.argtypes = pool * 2 + [I32] + [I64] * 4 + [P, I64, P, P, I64, P, P, I64, I64, P, SZ, P]
    lib.cfp32_cache_compact.restype = I32
    lib.cfp32_rotary_frequencies.argtypes = [F64, I64, I32] + [F64] * 4 + [P, P]
    lib.cfp32_rotary_frequencies.restype = I32
    lib.cfp32_rotary.argtypes = view * 2 + [I32, P, P, F64, I32, I32] + view * 2 + [I64] * 5 + [P]
    lib.cfp32_rotary.restype = I32
    lib.cfp32_cache8_append.argtypes = view * 2 + [P] * 5 + [I64] * 4 + [P]
    lib.cfp32_cache8_append.restype = I32
    lib.cfp32_cache8_read.argtypes = [P, P, I64, P, P] + view * 2 + [I32] + [I64] * 3 + [P]
    lib.cfp32_cache8_read.restype = I32
    lib.cfp32_cache8_copy_pages.argtypes = [P, P, P, I64, P]
    lib.cfp32_cache8_copy_pages.restype = I32
    lib.cfp32_cache8_fork.argtypes = [P, P, I64, P, P, P, P, I64, P, P, P] + [I64] * 3 + [P, SZ, P]
    lib.cfp32_cache8_fork.restype = I32
    lib.cfp32_cache8_compact.argtypes = [P, P, I64, P, P, I64, P, P, I64, I64, P, SZ, P]
    lib.cfp32_cache8_compact.restype = I32
    lib.cfp32_attention8_decode_workspace_bytes.argtypes = [I64] * 6
    lib.cfp32_attention8_decode_workspace_bytes.restype = SZ
    lib.cfp32_attention8_decode.argtypes = view + [P, P, I64, I64, P] + view + [I64, I64, F64, P, SZ, P]
    lib.cfp32_attention8_decode.restype = I32
    lib.cfp32_beam_select_workspace_bytes.argtypes = [I64] * 4
    lib.cfp32_beam_select_workspace_bytes.restype = SZ
    lib.cfp32_beam_select.argtypes = [P, I64, P, P] + [I64] * 5 + [P] * 5 + [SZ, P]
    lib.cfp32_beam_select.restype = I32
    lib.cfp32_beam_reorder.argtypes = [P, I64, P, I64, P, I64, I64, I64, P]
    lib.cfp32_beam_reorder.restype = I32
    _lib = lib
    return lib


# -- C entry points, same names, raw integers ------------------------------------

def cfp32_status_string(status: int) -> str:
    return load_library().cfp32_status_string(int(status)).decode()


def cfp32_last_hip_error() -> int:
    return int(load_library().cfp32_last_hip_error())


def cfp32_split(x, ldx, hi, lo, ldh, rows, cols, stream) -> int:
    return int(load_library().cfp32_split(x, ldx, hi, lo, ldh, rows, cols, stream))


def cfp32_gemm(a_hi, a_lo, lda, w, ldw, y, c_hi, c_lo, ldc, M, N, K, stream) -> int:
    return int(load_library().cfp32_gemm(a_hi, a_lo, lda, w, ldw, y, c_hi, c_lo, ldc, M, N, K, stream))


def cfp32_gemm_separate_add(a_hi, a_lo, lda, w, ldw, y, c_hi, c_lo, ldc, M, N, K, k_per_add, stream) -> int:
    return int(load_library().cfp32_gemm_separate_add(a_hi, a_lo, lda, w, ldw, y, c_hi, c_lo, ldc, M, N, K,
                                                      k_per_add, stream))


def cfp32_merge(c_hi, c_lo, ldc, y, ldy, M, N, stream) -> int:
    return int(load_library().cfp32_merge(c_hi, c_lo, ldc, y, ldy, M, N, stream))


def cfp32_linear_workspace_bytes(M, N, K) -> int:
    return int(load_library().cfp32_linear_workspace_bytes(M, N, K))


def cfp32_linear(x, ldx, w, ldw, y, ldy, M, N, K, workspace, workspace_bytes, stream) -> int:
    return int(load_library().cfp32_linear(x, ldx, w, ldw, y, ldy, M, N, K, workspace, workspace_bytes, stream))


def cfp32_linear_noalloc(x, ldx, w, ldw, y, ldy, M, N, K, stream) -> int:
    return int(load_library().cfp32_linear_noalloc(x, ldx, w, ldw, y, ldy, M, N, K, stream))


def cfp32_linear_ex_workspace_bytes(M, N, K, w_layout) -> int:
    return int(load_library().cfp32_linear_ex_workspace_bytes(M, N, K, w_layout))


def cfp32_linear_ex(x, ldx, w, ldw, w_layout, bias, y, ldy, M, N, K, workspace, workspace_bytes, stream) -> int:
    return int(load_library().cfp32_linear_ex(x, ldx, w, ldw, w_layout, bias, y, ldy, M, N, K, workspace,
                                              workspace_bytes, stream))


def cfp32_linear_geglu_workspace_bytes(M, F, K) -> int:
    return int(load_library().cfp32_linear_geglu_workspace_bytes(M, F, K))


def cfp32_linear_geglu(x, ldx, w, ldw, bias, out, ldo, M, F, K, workspace, workspace_bytes, stream) -> int:
    return int(load_library().cfp32_linear_geglu(x, ldx, w, ldw, bias, out, ldo, M, F, K, workspace,
                                                 workspace_bytes, stream))


def cfp32_linear_f32(x, ldx, w, ldw, y, ldy, M, N, K, stream) -> int:
    return int(load_library().cfp32_linear_f32(x, ldx, w, ldw, y, ldy, M, N, K, stream))


def cfp32_qkv_rotary(qkv, ldq, positions, theta, q, k, v, T, H, D, stream) -> int:
    return int(load_library().cfp32_qkv_rotary(qkv, ldq, positions, theta, q, k, v, T, H, D, stream))


def cfp32_attention_prompt_workspace_bytes(S, Tk, Hkv, D, kv_type) -> int:
    return int(load_library().cfp32_attention_prompt_workspace_bytes(S, Tk, Hkv, D, kv_type))


def cfp32_attention_prompt(q, q_tok, q_head, k, k_tok, k_head, v, v_tok, v_head, kv_type, cu_q, cu_k, out, out_tok,
                           out_head, S, Tq, Tk, Hq, Hkv, D, causal, scale, workspace, workspace_bytes, stream) -> int:
    return int(load_library().cfp32_attention_prompt(q, q_tok, q_head, k, k_tok, k_head, v, v_tok, v_head, kv_type,
                                                     cu_q, cu_k, out, out_tok, out_head, S, Tq, Tk, Hq, Hkv, D,
                                                     causal, scale, workspace, workspace_bytes, stream))


def cfp32_attention_decode_workspace_bytes(B, Hq, Hkv, D, W, page, shared_pages, kv_type) -> int:
    return int(load_library().cfp32_attention_decode_workspace_bytes(B, Hq, Hkv, D, W, page, shared_pages, kv_type))


def cfp32_attention_decode(q, q_seq, q_head, k_pages, k_page, k_head, k_tok, v_pages, v_page, v_head, v_tok, kv_type,
                           P, page, table, ld_table, W, lens, shared_pages, out, out_seq, out_head, B, Hq, Hkv, D,
                           scale, workspace, workspace_bytes, stream) -> int:
    return int(load_library().cfp32_attention_decode(q, q_seq, q_head, k_pages, k_page, k_head, k_tok, v_pages,
                                                     v_page, v_head, v_tok, kv_type, P, page, table, ld_table, W,
                                                     lens, shared_pages, out, out_seq, out_head, B, Hq, Hkv, D,
                                                     scale, workspace, workspace_bytes, stream))


def cfp32_cache_reserve(table, ld_table, lens, cu, refs, table_out, ld_out, refs_out, missing, S, W, P, page,
                        stream) -> int:
    return int(load_library().cfp32_cache_reserve(table, ld_table, lens, cu, refs, table_out, ld_out, refs_out,
                                                  missing, S, W, P, page, stream))


def cfp32_cache_append(k, k_tok, k_head, v, v_tok, v_head, cu, lens, lens_out, k_pages, kp_page, kp_head, kp_tok,
                       v_pages, vp_page, vp_head, vp_tok, kv_type, P, page, table, ld_table, S, W, T, Hkv, D,
                       stream) -> int:
    return int(load_library().cfp32_cache_append(k, k_tok, k_head, v, v_tok, v_head, cu, lens, lens_out, k_pages,
                                                 kp_page, kp_head, kp_tok, v_pages, vp_page, vp_head, vp_tok,
                                                 kv_type, P, page, table, ld_table, S, W, T, Hkv, D, stream))


def cfp32_cache_copy_pages(k_pages, kp_page, kp_head, kp_tok, v_pages, vp_page, vp_head, vp_tok, kv_type, P, page,
                           Hkv, D, src, dst, n, stream) -> int:
    return int(load_library().cfp32_cache_copy_pages(k_pages, kp_page, kp_head, kp_tok, v_pages, vp_page, vp_head,
                                                     vp_tok, kv_type, P, page, Hkv, D, src, dst, n, stream))


def cfp32_cache_fork_workspace_bytes(C) -> int:
    return int(load_library().cfp32_cache_fork_workspace_bytes(C))


def cfp32_cache_fork(k_pages, kp_page, kp_head, kp_tok, v_pages, vp_page, vp_head, vp_tok, kv_type, P, page, Hkv, D,
                     table, ld_table, lens, refs, parents, table_out, ld_out, lens_out, refs_out, missing, S, W, C,
                     workspace, workspace_bytes, stream) -> int:
    return int(load_library().cfp32_cache_fork(k_pages, kp_page, kp_head, kp_tok, v_pages, vp_page, vp_head, vp_tok,
                                               kv_type, P, page, Hkv, D, table, ld_table, lens, refs, parents,
                                               table_out, ld_out, lens_out, refs_out, missing, S, W, C, workspace,
                                               workspace_bytes, stream))


def cfp32_cache_free(rows, ld_rows, refs, refs_out, R, W, P, stream) -> int:
    return int(load_library().cfp32_cache_free(rows, ld_rows, refs, refs_out, R, W, P, stream))


def cfp32_cache_compact_workspace_bytes(P) -> int:
    return int(load_library().cfp32_cache_compact_workspace_bytes(P))


def cfp32_cache_compact(k_pages, kp_page, kp_head, kp_tok, v_pages, vp_page, vp_head, vp_tok, kv_type, P, page, Hkv,
                        D, table, ld_table, refs, table_out, ld_out, refs_out, live, S, W, workspace,
                        workspace_bytes, stream) -> int:
    return int(load_library().cfp32_cache_compact(k_pages, kp_page, kp_head, kp_tok, v_pages, vp_page, vp_head,
                                                  vp_tok, kv_type, P, page, Hkv, D, table, ld_table, refs, table_out,
                                                  ld_out, refs_out, live, S, W, workspace, workspace_bytes, stream))


def cfp32_rotary_frequencies(theta, R, scaling, factor, trained, slow, fast, frequencies, amplitude) -> int:
    return int(load_library().cfp32_rotary_frequencies(theta, R, scaling, factor, trained, slow, fast, frequencies,
                                                       amplitude))


def cfp32_rotary(q, q_tok, q_head, k, k_tok, k_head, type, positions, frequencies, amplitude, layout, transpose, q_out,
                 qo_tok, qo_head, k_out, ko_tok, ko_head, T, Hq, Hkv, D, R, stream) -> int:
    return int(load_library().cfp32_rotary(q, q_tok, q_head, k, k_tok, k_head, type, positions, frequencies, amplitude,
                                           layout, transpose, q_out, qo_tok, qo_head, k_out, ko_tok, ko_head, T, Hq,
                                           Hkv, D, R, stream))


def cfp32_cache8_append(k, k_tok, k_head, v, v_tok, v_head, cu, lens, lens_out, cache, table, ld_table, S, W, T,
                        stream) -> int:
    return int(load_library().cfp32_cache8_append(k, k_tok, k_head, v, v_tok, v_head, cu, lens, lens_out, cache, table,
                                                  ld_table, S, W, T, stream))


def cfp32_cache8_read(cache, table, ld_table, first, cu, k, k_tok, k_head, v, v_tok, v_head, out_type, S, W, T,
                      stream) -> int:
    return int(load_library().cfp32_cache8_read(cache, table, ld_table, first, cu, k, k_tok, k_head, v, v_tok, v_head,
                                                out_type, S, W, T, stream))


def cfp32_cache8_copy_pages(cache, src, dst, n, stream) -> int:
    return int(load_library().cfp32_cache8_copy_pages(cache, src, dst, n, stream))


def cfp32_cache8_fork(cache, table, ld_table, lens, refs, parents, table_out, ld_out, lens_out, refs_out, missing, S, W,
                      C, workspace, workspace_bytes, stream) -> int:
    return int(load_library().cfp32_cache8_fork(cache, table, ld_table, lens, refs, parents, table_out, ld_out, lens_out,
                                                refs_out, missing, S, W, C, workspace, workspace_bytes, stream))


def cfp32_cache8_compact(cache, table, ld_table, refs, table_out, ld_out, refs_out, live, S, W, workspace,
                         workspace_bytes, stream) -> int:
    return int(load_library().cfp32_cache8_compact(cache, table, ld_table, refs, table_out, ld_out, refs_out, live, S, W,
                                                   workspace, workspace_bytes, stream))


def cfp32_attention8_decode_workspace_bytes(B, Hq, Hkv, D, W, page) -> int:
    return int(load_library().cfp32_attention8_decode_workspace_bytes(B, Hq, Hkv, D, W, page))


def cfp32_attention8_decode(q, q_seq, q_head, cache, table, ld_table, W, lens, out, out_seq, out_head, B, Hq, scale,
                            workspace, workspace_bytes, stream) -> int:
    return int(load_library().cfp32_attention8_decode(q, q_seq, q_head, cache, table, ld_table, W, lens, out, out_seq,
                                                      out_head, B, Hq, scale, workspace, workspace_bytes, stream))


def cfp32_beam_select_workspace_bytes(S, beams, V, n) -> int:
    return int(load_library().cfp32_beam_select_workspace_bytes(S, beams, V, n))


def cfp32_beam_select(logits, ld, scores, done, S, beams, V, n, eos, parents, tokens, scores_out, done_out, workspace,
                      workspace_bytes, stream) -> int:
    return int(load_library().cfp32_beam_select(logits, ld, scores, done, S, beams, V, n, eos, parents, tokens, scores_out,
                                                done_out, workspace, workspace_bytes, stream))


def cfp32_beam_reorder(states, stride, out, out_stride, parents, rows, n, row_bytes, stream) -> int:
    return int(load_library().cfp32_beam_reorder(states, stride, out, out_stride, parents, rows, n, row_bytes, stream))


# -- tensor helpers -------------------------------------------------------------

def _torch():
    import torch
    return torch


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _row_step(t, name, shared=False):
    """Elements from one row of a 2-D tensor to the next, at least its columns; `shared`: or 0, all rows being one."""
    rows, cols = t.shape
    step = t.stride(0) if rows > 1 else cols
    if step < cols and not (shared and step == 0):
        raise ValueError(f"{name}: rows overlap (stride(0) is {step}, of {cols} columns)")
    return step


def _mat(t, dtypes, name, shared=False):
    """(pointer, rows, cols, ld) of a 2-D device tensor with unit column stride; `shared`: as ``_row_step`` has it."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name}: expected a GPU tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: columns must be contiguous (stride(1) == 1)")
    ld = _row_step(t, name, shared)
    return t.data_ptr(), rows, cols, ld if shared else max(ld, 1)


def _f16_dtypes():
    torch = _torch()
    d = [torch.float16, torch.int16]
    if hasattr(torch, "uint16"):
        d.append(torch.uint16)
    return tuple(d)


def _check(status, where):
    if status != OK:
        raise Cfp32Error(status, where)


def split(x, hi=None, lo=None, stream=None):
    """(hi, lo) = split(x): FP32 [rows, cols] -> two FP16 planes (float16)."""
    torch = _torch()
    px, rows, cols, ldx = _mat(x, (torch.float32,), "x")
    if hi is None:
        hi = torch.empty((rows, cols), dtype=torch.float16, device=x.device)
    if lo is None:
        lo = torch.empty((rows, cols), dtype=torch.float16, device=x.device)
    ph, r1, c1, ldh = _mat(hi, _f16_dtypes(), "hi")
    pl, r2, c2, ldl = _mat(lo, _f16_dtypes(), "lo")
    if (r1, c1) != (rows, cols) or (r2, c2) != (rows, cols) or ldh != ldl:
        raise ValueError("hi/lo must be [rows, cols] with one leading dimension")
    _check(cfp32_split(px, ldx, ph, pl, ldh, rows, cols, _stream(stream)), "cfp32_split")
    return hi, lo


def gemm(a_hi, a_lo, w, y=None, c_hi=None, c_lo=None, want_y=True, want_parts=False, stream=None):
    """Dual-product GEMM with fused merge.  Returns (y, c_hi, c_lo); entries not
    requested are None."""
    torch = _torch()
    pa, M, K, lda = _mat(a_hi, _f16_dtypes(), "a_hi")
    pb, M2, K2, lda2 = _mat(a_lo, _f16_dtypes(), "a_lo")
    pw, K3, N, ldw = _mat(w, _f16_dtypes(), "w")
    if (M2, K2) != (M, K) or lda2 != lda or K3 != K:
        raise ValueError("shape mismatch between a_hi, a_lo and w")
    dev = a_hi.device
    if want_y and y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=dev)
    if want_parts and c_hi is None:
        c_hi = torch.empty((M, N), dtype=torch.float32, device=dev)
        c_lo = torch.empty((M, N), dtype=torch.float32, device=dev)
    outs = [t for t in (y, c_hi, c_lo) if t is not None]
    lds = {(_mat(t, (torch.float32,), "out")[3]) for t in outs}
    if len(lds) != 1:
        raise ValueError("all outputs must share one leading dimension")
    ldc = lds.pop()
    py = y.data_ptr() if y is not None else None
    ph = c_hi.data_ptr() if c_hi is not None else None
    pl = c_lo.data_ptr() if c_lo is not None else None
    _check(cfp32_gemm(pa, pb, lda, pw, ldw, py, ph, pl, ldc, M, N, K, _stream(stream)), "cfp32_gemm")
    return y, c_hi, c_lo


def merge(c_hi, c_lo, y=None, stream=None):
    torch = _torch()
    ph, M, N, ldc = _mat(c_hi, (torch.float32,), "c_hi")
    pl, M2, N2, ldc2 = _mat(c_lo, (torch.float32,), "c_lo")
    if (M2, N2) != (M, N) or ldc2 != ldc:
        raise ValueError("c_hi and c_lo must match")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=c_hi.device)
    py, _, _, ldy = _mat(y, (torch.float32,), "y")
    _check(cfp32_merge(ph, pl, ldc, py, ldy, M, N, _stream(stream)), "cfp32_merge")
    return y


class Workspace:
    """Grow-only device scratch for the tensor helpers that take one.

    The library's kernels read and write the workspace asynchronously, in the
    order of the stream they are launched on, so one Workspace serves one
    stream at a time: calls on different streams that may overlap need one
    each (the helpers' default keeps one per device and stream).  A buffer is
    memory of the stream it is first handed to, so that what the allocator
    gave back for it is ordered with that stream's work, and is marked as used
    by every stream it is handed to (``record_stream``), so when it grows, the
    caching allocator does not give the old buffer to anyone else before the
    work queued on those streams is done.  Threads that launch on one stream
    may share one (their calls' kernels follow each other as a whole).  A call
    captured into a graph keeps the buffer's address: give it a Workspace of
    its own that lives as long as the graph and makes no larger calls."""

    def __init__(self):
        self.buf = None
        self._lock = threading.Lock()

    def get(self, nbytes, device, stream=None):
        if nbytes == 0:
            return None
        with self._lock:
            if self.buf is None or self.buf.numel() < nbytes or self.buf.device != device:
                self.buf = _empty(nbytes, _torch().uint8, device, stream)
            buf = self.buf
        if stream is not None:
            buf.record_stream(_on(stream))
        return buf


_default_lock = threading.Lock()
_default_ws: dict = {}


def _default_workspace(device, stream) -> Workspace:
    """The helpers' own workspace for (device, stream): calls on different
    streams never share scratch memory."""
    key = (device.index if device.index is not None else -1, _stream(stream))
    with _default_lock:
        ws = _default_ws.get(key)
        if ws is None:
            ws = _default_ws[key] = Workspace()
        return ws


def _stream_obj(stream):
    """The torch stream a helper call runs on (the current one by default)."""
    if stream is None:
        return _torch().cuda.current_stream()
    return stream


def linear(x, w, out=None, workspace: Workspace | None = None, stream=None, bias=None, w_layout: str = "kn"):
    """y = x W (+ bias) with the compensated-FP32 method: x FP32 [M,K]; w FP16
    [K,N] (w_layout "kn") or [N,K] ("nk", a torch.nn.Linear weight); bias
    FP32 [N] or None."""
    torch = _torch()
    if w_layout not in ("kn", "nk"):
        raise ValueError("w_layout must be 'kn' or 'nk'")
    px, M, K, ldx = _mat(x, (torch.float32,), "x")
    pw, r, c, ldw = _mat(w, _f16_dtypes(), "w")
    K2, N = (r, c) if w_layout == "kn" else (c, r)
    if K2 != K:
        raise ValueError("inner dimensions differ")
    pb = None
    if bias is not None:
        if bias.dtype != torch.float32 or bias.device != x.device or bias.dim() != 1 or bias.shape[0] != N \
                or (N > 1 and bias.stride(0) != 1):
            raise ValueError("bias must be a contiguous FP32 [N] tensor on x's device")
        pb = bias.data_ptr()
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=x.device)
    py, M3, N3, ldy = _mat(out, (torch.float32,), "out")
    if (M3, N3) != (M, N):
        raise ValueError("out has the wrong shape")
    layout = W_KN if w_layout == "kn" else W_NK
    need = cfp32_linear_ex_workspace_bytes(M, N, K, layout)
    st = _stream_obj(stream)
    ws = (workspace or _default_workspace(x.device, st)).get(need, x.device, st)
    pws = ws.data_ptr() if ws is not None else None
    _check(cfp32_linear_ex(px, ldx, pw, ldw, layout, pb, py, ldy, M, N, K, pws, need, _stream(st)),
           "cfp32_linear_ex")
    return out


def linear_geglu(x, w, bias=None, out=None, workspace: Workspace | None = None, stream=None):
    """out = gelu(x W[:, :F] + b[:F]) * (x W[:, F:] + b[F:]): x FP32 [M,K], w FP16
    [K, 2F] (gate columns, then up columns), bias FP32 [2F] or None."""
    torch = _torch()
    px, M, K, ldx = _mat(x, (torch.float32,), "x")
    pw, K2, N2, ldw = _mat(w, _f16_dtypes(), "w")
    if K2 != K or N2 % 2:
        raise ValueError("w must be [K, 2F]")
    F = N2 // 2
    pb = None
    if bias is not None:
        if bias.dtype != torch.float32 or bias.device != x.device or bias.dim() != 1 or bias.shape[0] != 2 * F \
                or (F > 0 and bias.stride(0) != 1):
            raise ValueError("bias must be a contiguous FP32 [2F] tensor on x's device")
        pb = bias.data_ptr()
    if out is None:
        out = torch.empty((M, F), dtype=torch.float32, device=x.device)
    po, M3, F3, ldo = _mat(out, (torch.float32,), "out")
    if (M3, F3) != (M, F):
        raise ValueError("out has the wrong shape")
    need = cfp32_linear_geglu_workspace_bytes(M, F, K)
    st = _stream_obj(stream)
    ws = (workspace or _default_workspace(x.device, st)).get(need, x.device, st)
    pws = ws.data_ptr() if ws is not None else None
    _check(cfp32_linear_geglu(px, ldx, pw, ldw, pb, po, ldo, M, F, K, pws, need, _stream(st)),
           "cfp32_linear_geglu")
    return out


def linear_f32(x, w, out=None, stream=None):
    """The true-FP32 projection y = x W: x FP32 [M, K] used as FP32, w FP16
    [K, N] widened exactly, FP32 matrix-unit products and sums."""
    torch = _torch()
    px, M, K, ldx = _mat(x, (torch.float32,), "x")
    pw, K2, N, ldw = _mat(w, _f16_dtypes(), "w")
    if K2 != K:
        raise ValueError("inner dimensions differ")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=x.device)
    py, M3, N3, ldy = _mat(out, (torch.float32,), "out")
    if (M3, N3) != (M, N):
        raise ValueError("out has the wrong shape")
    _check(cfp32_linear_f32(px, ldx, pw, ldw, py, ldy, M, N, K, _stream(stream)), "cfp32_linear_f32")
    return out


def qkv_rotary(qkv, H: int, D: int, positions=None, theta: float = 10000.0, stream=None):
    """(q, k, v), each FP32 [H, T, D], from a QKV projection output [T, 3 H D]
    (row t = [q | k | v]); q and k rotated (half-split pairs), v copied."""
    torch = _torch()
    pq, T, C, ldq = _mat(qkv, (torch.float32,), "qkv")
    if C < 3 * H * D:
        raise ValueError("qkv has fewer than 3*H*D columns")
    pp = None
    if positions is not None:
        if positions.dtype != torch.int64 or positions.device != qkv.device or positions.numel() != T \
                or not positions.is_contiguous():
            raise ValueError("positions must be a contiguous int64 [T] tensor on qkv's device")
        pp = positions.data_ptr()
    q, k, v = (torch.empty((H, T, D), dtype=torch.float32, device=qkv.device) for _ in range(3))
    _check(cfp32_qkv_rotary(pq, ldq, pp, float(theta), q.data_ptr(), k.data_ptr(), v.data_ptr(), T, H, D,
                            _stream(stream)), "cfp32_qkv_rotary")
    return q, k, v


# -- attention and the paged cache ----------------------------------------------

_helpers = None


class _NoNative:
    """In the place of the helpers' native form: declines every call."""

    def __getattr__(self, name):
        return lambda *args: None


def _native():
    """The helpers' native form (csrc/helpers.cpp), bound to the loaded library;
    where it was not built, the calls are made from Python."""
    global _helpers
    if _helpers is None:
        torch = _torch()
        import importlib.util
        path = os.path.join(_HERE, "_helpers.so")
        try:
            spec = importlib.util.spec_from_file_location(__name__ + "._helpers", path)
            mod = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(mod)
        except ImportError as e:
            import warnings
            warnings.warn(f"the native form of the attention and cache helpers is not there ({e}): their calls take "
                          "10 to 15 us more of host time", RuntimeWarning, stacklevel=3)
            _helpers = _NoNative()
            return _helpers
        lib = load_library()
        names = ("cfp32_attention_prompt_workspace_bytes", "cfp32_attention_prompt",
                 "cfp32_attention_decode_workspace_bytes", "cfp32_attention_decode", "cfp32_cache_reserve",
                 "cfp32_cache_append", "cfp32_cache_fork_workspace_bytes", "cfp32_cache_fork", "cfp32_cache_free",
                 "cfp32_cache_compact_workspace_bytes", "cfp32_cache_compact", "cfp32_rotary", "cfp32_cache8_append",
                 "cfp32_cache8_read", "cfp32_attention8_decode_workspace_bytes", "cfp32_attention8_decode",
                 "cfp32_beam_select_workspace_bytes", "cfp32_beam_select", "cfp32_beam_reorder")
        mod.bind(tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names),
                 torch._C._cuda_getCurrentRawStream, _scratch_buffer)
        _helpers = mod
    return _helpers


def _scratch_buffer(need, index, raw):
    """The helpers' own workspace for the current stream `raw` of device
    `index`, for the native form; None where it has to be allocated first."""
    ws = _default_ws.get((index, raw))
    buf = None if ws is None else ws.buf
    return None if buf is None or buf.numel() < need else buf


def _heads(t, dtypes, name, device):
    """(pointer, token stride, head stride) of a [tokens, heads, D] tensor with unit stride along D."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name}: expected a GPU tensor")
    if t.device != device:
        raise ValueError(f"{name}: on another device")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.dim() != 3:
        raise ValueError(f"{name}: expected a 3-D tensor")
    a, b, c = t.stride()
    if c != 1 and t.shape[2] > 1 and t.numel():
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), a, b


def _ints(t, name, device, dim):
    """Pointer of an int32 tensor: contiguous along its last dimension."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != device:
        raise TypeError(f"{name}: expected an int32 tensor on {device}")
    if t.dim() != dim or (t.shape[-1] > 1 and t.stride(-1) != 1 and t.numel()):
        raise ValueError(f"{name}: expected a {dim}-D tensor with contiguous rows")
    return t.data_ptr()


def _ld(t, name="table", shared=False):
    return _row_step(t, name, shared)


def _pools(k_pages, v_pages):
    """(K and V as pointer and page, head and token strides), kv_type and shape of a pair of pools."""
    torch = _torch()
    at = []
    for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
            raise TypeError(f"{name}: expected a GPU tensor")
        if t.dtype not in (torch.float32, torch.float16):
            raise TypeError(f"{name}: dtype {t.dtype} is neither float32 nor float16")
        if t.dim() != 4 or (t.shape[3] > 1 and t.stride(3) != 1 and t.numel()):
            raise ValueError(f"{name}: expected [pages, heads, tokens, D] with contiguous D")
        at += [t.data_ptr(), *t.stride()[:3]]
    if k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype or k_pages.device != v_pages.device:
        raise ValueError("k_pages and v_pages differ in shape, dtype or device")
    return at, KV_F16 if k_pages.dtype == torch.float16 else KV_F32, k_pages.shape


def _on(stream):
    """The torch stream of a helper call (an integer handle is wrapped)."""
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream()
    return stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream))


def _empty(shape, dtype, device, stream):
    """A new tensor in the memory of the stream that writes it, so that the
    allocator's reuse is ordered with the work queued there."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_on(stream)):
        return torch.empty(shape, dtype=dtype, device=device)


def _scratch(need, device, workspace, stream):
    """(buffer, its address, stream handle) of a call; the buffer is held until
    the call is made (another thread's may make the workspace grow meanwhile)."""
    st = _on(stream)
    if not need:
        return None, None, _stream(st)
    buf = (workspace or _default_workspace(device, st)).get(need, device, st)
    return buf, buf.data_ptr(), _stream(st)


def attention_prompt(q, k, v, cu_q, cu_k=None, causal: bool = True, scale: float | None = None, out=None,
                     workspace: Workspace | None = None, stream=None):
    """Attention over packed prompts: q FP32 [Tq, Hq, D]; k, v FP32 or FP16
    [Tk, Hkv, D] (any strides with contiguous D: pass ``qkv_rotary``'s
    [H, T, D] as ``.transpose(0, 1)``); cu_q, cu_k int32 [S + 1] offsets of
    the sequences (cu_k defaults to cu_q).  Causal rows are aligned to the
    end of their sequence's keys.  scale defaults to 1 / sqrt(D).  Returns
    FP32 [Tq, Hq, D]; rows outside all sequences are not written."""
    if stream is None and workspace is None:
        done = _native().attention_prompt(q, k, v, cu_q, cu_k, causal, scale, out)
        if done is not None:
            return done
    torch = _torch()
    pq = _heads(q, (torch.float32,), "q", q.device)
    dev = q.device
    pk = _heads(k, (torch.float32, torch.float16), "k", dev)
    pv = _heads(v, (k.dtype,), "v", dev)
    Tq, Hq, D = q.shape
    Tk, Hkv, D2 = k.shape
    if v.shape != k.shape or D2 != D or Hkv == 0 or Hq % Hkv:
        raise ValueError("shape mismatch between q, k and v")
    cu_k = cu_q if cu_k is None else cu_k
    cq, ck = _ints(cu_q, "cu_q", dev, 1), _ints(cu_k, "cu_k", dev, 1)
    S = cu_q.shape[0] - 1
    if S < 0 or cu_k.shape[0] != S + 1:
        raise ValueError("cu_q and cu_k must both have one entry more than there are sequences")
    if out is None:
        out = _empty((Tq, Hq, D), torch.float32, dev, stream)
    elif out.shape != q.shape:
        raise ValueError("out has the wrong shape")
    po = _heads(out, (torch.float32,), "out", dev)
    kv = KV_F16 if k.dtype == torch.float16 else KV_F32
    need = cfp32_attention_prompt_workspace_bytes(S, Tk, Hkv, D, kv)
    buf, ws, st = _scratch(need, dev, workspace, stream)
    _check(cfp32_attention_prompt(*pq, *pk, *pv, kv, cq, ck, *po, S, Tq, Tk, Hq, Hkv, D, 1 if causal else 0,
                                  D ** -0.5 if scale is None else scale, ws, need, st), "cfp32_attention_prompt")
    return out


def attention_decode(q, k_pages, v_pages, table, lens, shared_pages: int = 0, scale: float | None = None, out=None,
                     workspace: Workspace | None = None, stream=None):
    """Attention of one new token per sequence against a paged cache: q FP32
    [B, Hq, D]; pools [P, Hkv, page, D]; table int32 [B, W]; lens int32 [B].
    The first ``shared_pages`` table entries are the same in every row and
    are read once for the batch.  Returns FP32 [B, Hq, D]."""
    if stream is None and workspace is None:
        done = _native().attention_decode(q, k_pages, v_pages, table, lens, shared_pages, scale, out)
        if done is not None:
            return done
    torch = _torch()
    dev = q.device
    pq = _heads(q, (torch.float32,), "q", dev)
    at, kv, (P, Hkv, page, D2) = _pools(k_pages, v_pages)
    B, Hq, D = q.shape
    if k_pages.device != dev or D2 != D or Hkv == 0 or Hq % Hkv:
        raise ValueError("q and the pools differ in head size, heads or device")
    pt, pl = _ints(table, "table", dev, 2), _ints(lens, "lens", dev, 1)
    W = table.shape[1]
    if table.shape[0] != B or lens.shape[0] != B:
        raise ValueError("table and lens must have one row per sequence")
    if out is None:
        out = _empty((B, Hq, D), torch.float32, dev, stream)
    elif out.shape != q.shape:
        raise ValueError("out has the wrong shape")
    po = _heads(out, (torch.float32,), "out", dev)
    need = cfp32_attention_decode_workspace_bytes(B, Hq, Hkv, D, W, page, shared_pages, kv)
    buf, ws, st = _scratch(need, dev, workspace, stream)
    _check(cfp32_attention_decode(*pq, *at, kv, P, page, pt, _ld(table, shared=True), W, pl, shared_pages, *po, B, Hq, Hkv, D,
                                  D ** -0.5 if scale is None else scale, ws, need, st), "cfp32_attention_decode")
    return out


def cache_reserve(table, lens, refs, cu, page: int, missing=None, table_out=None, refs_out=None, stream=None):
    """(table, refs) with the lowest free pages in the entries that the new
    tokens need: sequence s holds lens[s] tokens and gets cu[s+1] - cu[s]
    more.  ``missing`` (int32 [1]) receives how many pages could not be given."""
    if stream is None and missing is None and table_out is None and refs_out is None:
        done = _native().cache_reserve(table, lens, refs, cu, page)
        if done is not None:
            return done
    torch = _torch()
    dev = table.device
    pt, pl, pr, pc = (_ints(table, "table", dev, 2), _ints(lens, "lens", dev, 1), _ints(refs, "refs", dev, 1),
                      _ints(cu, "cu", dev, 1))
    S, W = table.shape
    if lens.shape[0] != S or cu.shape[0] != S + 1:
        raise ValueError("lens must have one entry per sequence, cu one more")
    table_out = _empty((S, W), torch.int32, dev, stream) if table_out is None else table_out
    refs_out = _empty(refs.shape, torch.int32, dev, stream) if refs_out is None else refs_out
    pto, pro = _ints(table_out, "table_out", dev, 2), _ints(refs_out, "refs_out", dev, 1)
    pm = None if missing is None else _ints(missing, "missing", dev, 1)
    if table_out.shape != table.shape or refs_out.shape != refs.shape or (missing is not None and not missing.numel()):
        raise ValueError("table_out, refs_out or missing has the wrong shape")
    _check(cfp32_cache_reserve(pt, _ld(table), pl, pc, pr, pto, _ld(table_out, "table_out"), pro, pm, S, W, refs.shape[0], page,
                               _stream(stream)), "cfp32_cache_reserve")
    return table_out, refs_out


def cache_append(k, v, cu, k_pages, v_pages, table, lens, lens_out=None, stream=None):
    """Writes new tokens, k and v FP32 [T, Hkv, D], into the pools (rounded to
    their type): rows cu[s] .. cu[s+1] - 1 become tokens lens[s], ... of
    sequence s.  Returns the new lengths."""
    if stream is None and lens_out is None:
        done = _native().cache_append(k, v, cu, k_pages, v_pages, table, lens)
        if done is not None:
            return done
    torch = _torch()
    at, kv, (P, Hkv, page, D) = _pools(k_pages, v_pages)
    dev = k_pages.device
    pk, pv = _heads(k, (torch.float32,), "k", dev), _heads(v, (torch.float32,), "v", dev)
    if k.shape != v.shape or k.shape[1] != Hkv or k.shape[2] != D:
        raise ValueError("k, v and the pools differ in heads or head size")
    pt, pl, pc = _ints(table, "table", dev, 2), _ints(lens, "lens", dev, 1), _ints(cu, "cu", dev, 1)
    S, W = table.shape
    if lens.shape[0] != S or cu.shape[0] != S + 1:
        raise ValueError("lens must have one entry per sequence, cu one more")
    lens_out = _empty(lens.shape, torch.int32, dev, stream) if lens_out is None else lens_out
    plo = _ints(lens_out, "lens_out", dev, 1)
    if lens_out.shape != lens.shape:
        raise ValueError("lens_out has the wrong shape")
    _check(cfp32_cache_append(*pk, *pv, pc, pl, plo, *at, kv, P, page, pt, _ld(table), S, W, k.shape[0], Hkv, D,
                              _stream(stream)), "cfp32_cache_append")
    return lens_out


def cache_copy_pages(k_pages, v_pages, src, dst, stream=None):
    """Copies page src[i] of both pools to page dst[i] (int32 [n] each)."""
    at, kv, (P, Hkv, page, D) = _pools(k_pages, v_pages)
    dev = k_pages.device
    ps, pd = _ints(src, "src", dev, 1), _ints(dst, "dst", dev, 1)
    if src.shape != dst.shape:
        raise ValueError("src and dst differ in length")
    _check(cfp32_cache_copy_pages(*at, kv, P, page, Hkv, D, ps, pd, src.shape[0], _stream(stream)),
           "cfp32_cache_copy_pages")


def cache_fork(k_pages, v_pages, table, lens, refs, parents, missing=None, refs_out=None,
               workspace: Workspace | None = None, stream=None):
    """(table, refs, lens) of children of running sequences: child c shares the
    whole pages of sequence parents[c] and gets a copy of its partly filled
    last page.  ``missing`` (int32 [1]) receives how many last pages the pool
    had no page for."""
    if stream is None and workspace is None and missing is None and refs_out is None:
        done = _native().cache_fork(k_pages, v_pages, table, lens, refs, parents)
        if done is not None:
            return done
    torch = _torch()
    at, kv, (P, Hkv, page, D) = _pools(k_pages, v_pages)
    dev = k_pages.device
    pt, pl, pr, pp = (_ints(table, "table", dev, 2), _ints(lens, "lens", dev, 1), _ints(refs, "refs", dev, 1),
                      _ints(parents, "parents", dev, 1))
    (S, W), C = table.shape, parents.shape[0]
    if lens.shape[0] != S or refs.shape[0] != P:
        raise ValueError("lens must have one entry per sequence, refs one per page")
    table_out = _empty((C, W), torch.int32, dev, stream)
    lens_out = _empty(C, torch.int32, dev, stream)
    refs_out = _empty(refs.shape, torch.int32, dev, stream) if refs_out is None else refs_out
    pro = _ints(refs_out, "refs_out", dev, 1)
    pm = None if missing is None else _ints(missing, "missing", dev, 1)
    if refs_out.shape != refs.shape or (missing is not None and not missing.numel()):
        raise ValueError("refs_out or missing has the wrong shape")
    need = cfp32_cache_fork_workspace_bytes(C)
    buf, ws, st = _scratch(need, dev, workspace, stream)
    _check(cfp32_cache_fork(*at, kv, P, page, Hkv, D, pt, _ld(table), pl, pr, pp, table_out.data_ptr(), W,
                            lens_out.data_ptr(), pro, pm, S, W, C, ws, need, st), "cfp32_cache_fork")
    return table_out, refs_out, lens_out


def cache_free(rows, refs, refs_out=None, stream=None):
    """refs with the pages named in rows [R, W] (tables of ended sequences) given up."""
    if stream is None and refs_out is None:
        done = _native().cache_free(rows, refs)
        if done is not None:
            return done
    torch = _torch()
    dev = refs.device
    pw, pr = _ints(rows, "rows", dev, 2), _ints(refs, "refs", dev, 1)
    refs_out = _empty(refs.shape, torch.int32, dev, stream) if refs_out is None else refs_out
    pro = _ints(refs_out, "refs_out", dev, 1)
    if refs_out.shape != refs.shape:
        raise ValueError("refs_out has the wrong shape")
    R, W = rows.shape
    _check(cfp32_cache_free(pw, _ld(rows, "rows"), pr, pro, R, W, refs.shape[0], _stream(stream)), "cfp32_cache_free")
    return refs_out


def cache_compact(k_pages, v_pages, table, refs, table_out=None, refs_out=None, workspace: Workspace | None = None,
                  stream=None):
    """(table, refs, n) of the pool made dense: its n live pages are moved to
    pages 0 .. n - 1, and the table names them there.  n is an int32 [1] tensor."""
    if stream is None and workspace is None and table_out is None and refs_out is None:
        done = _native().cache_compact(k_pages, v_pages, table, refs)
        if done is not None:
            return done
    torch = _torch()
    at, kv, (P, Hkv, page, D) = _pools(k_pages, v_pages)
    dev = k_pages.device
    pt, pr = _ints(table, "table", dev, 2), _ints(refs, "refs", dev, 1)
    S, W = table.shape
    if refs.shape[0] != P:
        raise ValueError("refs must have one entry per page")
    table_out = _empty((S, W), torch.int32, dev, stream) if table_out is None else table_out
    refs_out = _empty(refs.shape, torch.int32, dev, stream) if refs_out is None else refs_out
    pto, pro = _ints(table_out, "table_out", dev, 2), _ints(refs_out, "refs_out", dev, 1)
    if table_out.shape != table.shape or refs_out.shape != refs.shape:
        raise ValueError("table_out or refs_out has the wrong shape")
    live = _empty(1, torch.int32, dev, stream)
    need = cfp32_cache_compact_workspace_bytes(P)
    buf, ws, st = _scratch(need, dev, workspace, stream)
    _check(cfp32_cache_compact(*at, kv, P, page, Hkv, D, pt, _ld(table), pr, pto, _ld(table_out, "table_out"), pro,
                               live.data_ptr(), S, W, ws, need, st), "cfp32_cache_compact")
    return table_out, refs_out, live


# -- rotary positions --------------------------------------------------------------

_SCALINGS = {"plain": ROTARY_PLAIN, "linear": ROTARY_LINEAR, "ntk": ROTARY_NTK, "parts": ROTARY_PARTS}


def _launch(call, where, device, *args, stream=None):
    """The call on `stream`, or the current stream of `device`, with that device current."""
    torch = _torch()
    with torch.cuda.device(device):
        _check(call(*args, _stream(stream)), where)


def rotary_frequencies(rotary_dim: int, theta: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                       trained: float = 0.0, slow: float = 1.0, fast: float = 32.0, device="cuda"):
    """(frequencies, amplitude) for ``rotary``: the angle each of the
    rotary_dim / 2 pairs turns by from one position to the next, FP64 on
    `device`, and the factor on the turned values.  scaling: "plain",
    "linear" (positions divided by `factor`), "ntk" (a larger base) or
    "parts" (pairs of fewer than `slow` turns within the `trained` length
    are interpolated, of more than `fast` left, between them in part)."""
    torch = _torch()
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    f = (ctypes.c_double * max(rotary_dim // 2, 1))()
    amplitude = ctypes.c_double()
    _check(cfp32_rotary_frequencies(float(theta), rotary_dim, _SCALINGS[scaling], float(factor), float(trained), float(slow),
                                    float(fast), f, ctypes.byref(amplitude)), "cfp32_rotary_frequencies")
    return torch.tensor(list(f), dtype=torch.float64, device=device), amplitude.value


def rotary(q, k, frequencies, positions=None, layout: str = "half", amplitude: float = 1.0, transpose: bool = False,
           q_out=None, k_out=None, stream=None):
    """(q, k) turned by their tokens' positions: q [T, Hq, D] and k [T, Hkv, D]
    (or None), FP32 or FP16, any strides with contiguous D; frequencies FP64
    [R / 2] for the first R dims; positions int64 [T] (0 .. T-1 if None).
    layout: "half" (pairs i, i + R/2) or "interleaved" (2i, 2i + 1).
    ``transpose`` takes gradients of the outputs to those of the inputs (as
    all calls here, it records no graph for autograd).
    q_out and k_out may be q and k, in this order, and overlap nothing else."""
    if layout not in ("half", "interleaved"):
        raise ValueError("layout must be 'half' or 'interleaved'")
    if stream is None:
        done = _native().rotary(q, k, frequencies, positions, layout == "interleaved", amplitude, transpose, q_out, k_out)
        if done is not None:
            return done
    torch = _torch()
    if not isinstance(q, torch.Tensor) or q.device.type != "cuda":
        raise TypeError("q: expected a GPU tensor")
    dev, types = q.device, (torch.float32, torch.float16)
    pq = _heads(q, types, "q", dev)
    T, Hq, D = q.shape
    pk, Hkv = (None, 0, 0), 0
    if k is not None:
        pk, Hkv = _heads(k, (q.dtype,), "k", dev), k.shape[1]
        if k.shape[0] != T or k.shape[2] != D:
            raise ValueError("q and k differ in tokens or head size")
    if not isinstance(frequencies, torch.Tensor) or frequencies.dtype != torch.float64 or frequencies.device != dev or \
            frequencies.dim() != 1 or not frequencies.is_contiguous() or 2 * frequencies.shape[0] > D:
        raise ValueError("frequencies must be a contiguous FP64 tensor of at most D / 2 values on q's device")
    pp = None
    if positions is not None:
        if positions.dtype != torch.int64 or positions.device != dev or positions.shape != (T,) or \
                not positions.is_contiguous():
            raise ValueError("positions must be a contiguous int64 [T] tensor on q's device")
        pp = positions.data_ptr()
    outs = []
    for x, out, name in ((q, q_out, "q_out"), (k, k_out, "k_out")):
        if x is None:
            outs.append(None)
            continue
        out = _empty(x.shape, x.dtype, dev, stream) if out is None else out
        if out.shape != x.shape:
            raise ValueError(f"{name} has the wrong shape")
        outs.append(out)
    po = _heads(outs[0], (q.dtype,), "q_out", dev)
    pko = (None, 0, 0) if k is None else _heads(outs[1], (q.dtype,), "k_out", dev)
    if T * Hq * Hkv * D and (po[0] in (pk[0], pko[0]) or pko[0] == pq[0]):
        raise ValueError("q_out and k_out may be q and k, in this order, and nothing that the other is")
    _launch(cfp32_rotary, "cfp32_rotary", dev, *pq, *pk, KV_F16 if q.dtype == torch.float16 else KV_F32, pp,
            frequencies.data_ptr(), float(amplitude), ROTARY_INTERLEAVED if layout == "interleaved" else ROTARY_HALF,
            1 if transpose else 0, *po, *pko, T, Hq, Hkv, D, 2 * frequencies.shape[0], stream=stream)
    return outs[0], outs[1]


# -- the 8-bit cache -----------------------------------------------------------------

class Cache8:
    """The pools of an 8-bit cache: codes k, v [P, Hkv, page, D] (int8 or
    float8_e4m3fn, any strides with contiguous D) and FP32 scales [P, Hkv,
    page / block], one for each block of tokens and head (``blocks`` of a
    page: powers of two).  The calls read and write the memory of the tensors
    that it is made of, which it keeps, whatever becomes of those: its
    attributes are not to be set, nor their storages resized."""

    __slots__ = ("k", "v", "k_scales", "v_scales", "desc", "addr", "device", "index", "shape", "block", "_held")

    def __setattr__(self, name, value):
        if hasattr(self, name):
            raise AttributeError(f"{name}: the pools of a Cache8 are those it was made of")
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        raise AttributeError(f"{name}: the pools of a Cache8 are those it was made of")

    def __init__(self, k, v, k_scales, v_scales):
        torch = _torch()
        for t, name in ((k, "k"), (v, "v"), (k_scales, "k_scales"), (v_scales, "v_scales")):
            if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
                raise TypeError(f"{name}: expected a GPU tensor")
            if t.device != k.device:
                raise ValueError(f"{name}: on another device")
        for t, name in ((k, "k"), (v, "v")):
            if t.dtype not in (torch.int8, torch.float8_e4m3fn) or t.dtype != k.dtype:
                raise TypeError(f"{name}: codes must be int8 or float8_e4m3fn, K and V alike")
            if t.dim() != 4 or t.shape != k.shape or (t.shape[3] > 1 and t.stride(3) != 1 and t.numel()):
                raise ValueError(f"{name}: expected [pages, heads, tokens, D] with contiguous D, K and V alike")
        P, Hkv, page, D = k.shape
        for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            if t.dtype != torch.float32:
                raise TypeError(f"{name}: scales must be float32")
            if t.dim() != 3 or t.shape != k_scales.shape or t.shape[:2] != (P, Hkv) or \
                    (t.shape[2] > 1 and t.stride(2) != 1 and t.numel()):
                raise ValueError(f"{name}: expected [pages, heads, blocks of a page] with contiguous blocks")
        blocks = k_scales.shape[2]
        if blocks < 1 or page % blocks or page & (page - 1) or blocks & (blocks - 1) or not 1 <= page <= 65536:
            raise ValueError("tokens and blocks of a page must be powers of two, of at most 65536 tokens")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        # What `desc` points to: of a tensor that is given another storage, the old one stays here.
        self._held = tuple(t.detach() for t in (k, v, k_scales, v_scales))
        self.device, self.shape, self.block = k.device, k.shape, page // blocks
        self.desc = Cache8Desc(k.data_ptr(), v.data_ptr(), *k.stride()[:3], *v.stride()[:3], k_scales.data_ptr(),
                               v_scales.data_ptr(), *k_scales.stride()[:2], *v_scales.stride()[:2], P, Hkv, page,
                               self.block, D, CODE_I8 if k.dtype == torch.int8 else CODE_E4M3)
        self.addr, self.index = ctypes.addressof(self.desc), k.device.index

    @classmethod
    def empty(cls, pages: int, heads: int, page: int, dim: int, block: int | None = None, dtype=None, device="cuda"):
        """Pools of their own, with nothing in them; a block of tokens is a page unless given."""
        torch = _torch()
        block = page if block is None else block
        if block < 1 or page % block:
            raise ValueError("block must divide page")
        codes = [torch.zeros((pages, heads, page, dim), dtype=torch.int8, device=device).view(dtype or torch.int8)
                 for _ in range(2)]
        return cls(*codes, *(torch.zeros((pages, heads, page // block), dtype=torch.float32, device=device) for _ in range(2)))


def _cache8(cache):
    if not isinstance(cache, Cache8):
        raise TypeError("cache: expected a Cache8")
    return cache


def cache8_append(k, v, cu, cache: Cache8, table, lens, lens_out=None, stream=None):
    """Writes new tokens, k and v FP32 [T, Hkv, D], into an 8-bit cache, as
    ``cache_append``: rows cu[s] .. cu[s+1] - 1 become tokens lens[s], ... of
    sequence s.  Returns the new lengths."""
    P, Hkv, page, D = _cache8(cache).shape
    if stream is None and lens_out is None:
        done = _native().cache8_append(k, v, cu, cache.addr, cache.index, table, lens)
        if done is not None:
            return done
    dev = cache.device
    torch = _torch()
    pk, pv = _heads(k, (torch.float32,), "k", dev), _heads(v, (torch.float32,), "v", dev)
    if k.shape != v.shape or k.shape[1] != Hkv or k.shape[2] != D:
        raise ValueError("k, v and the pools differ in heads or head size")
    pt, pl, pc = _ints(table, "table", dev, 2), _ints(lens, "lens", dev, 1), _ints(cu, "cu", dev, 1)
    S, W = table.shape
    if lens.shape[0] != S or cu.shape[0] != S + 1:
        raise ValueError("lens must have one entry per sequence, cu one more")
    lens_out = _empty(lens.shape, torch.int32, dev, stream) if lens_out is None else lens_out
    plo = _ints(lens_out, "lens_out", dev, 1)
    if lens_out.shape != lens.shape:
        raise ValueError("lens_out has the wrong shape")
    _launch(cfp32_cache8_append, "cfp32_cache8_append", dev, *pk, *pv, pc, pl, plo, cache.addr, pt, _ld(table), S, W,
            k.shape[0], stream=stream)
    return lens_out


def cache8_read(cache: Cache8, table, cu, tokens: int, first=None, dtype=None, k_out=None, v_out=None, stream=None):
    """(k, v), [tokens, Hkv, D] of `dtype` (FP32 or FP16), read back from an
    8-bit cache as ``attention_prompt`` takes them: rows cu[s] .. cu[s+1] - 1
    are tokens first[s], first[s] + 1, ... of sequence s (from 0 on without
    ``first``).  `tokens` is cu's last entry, or more: rows beyond it are not
    written."""
    torch = _torch()
    P, Hkv, page, D = _cache8(cache).shape
    dev = cache.device
    dtype = torch.float32 if dtype is None else dtype
    if dtype not in (torch.float32, torch.float16):
        raise TypeError("dtype must be float32 or float16")
    if stream is None and k_out is None and v_out is None:
        done = _native().cache8_read(cache.addr, cache.index, table, cu, tokens, first, dtype == torch.float16)
        if done is not None:
            return done
    pt, pc = _ints(table, "table", dev, 2), _ints(cu, "cu", dev, 1)
    S, W = table.shape
    pf = None if first is None else _ints(first, "first", dev, 1)
    if cu.shape[0] != S + 1 or (first is not None and first.shape[0] != S):
        raise ValueError("first must have one entry per sequence, cu one more")
    outs = []
    for out, name in ((k_out, "k_out"), (v_out, "v_out")):
        out = _empty((tokens, Hkv, D), dtype, dev, stream) if out is None else out
        if out.shape != (tokens, Hkv, D):
            raise ValueError(f"{name} has the wrong shape")
        outs.append(out)
    pk, pv = (_heads(o, (dtype,), n, dev) for o, n in zip(outs, ("k_out", "v_out")))
    _launch(cfp32_cache8_read, "cfp32_cache8_read", dev, cache.addr, pt, _ld(table, shared=True), pf, pc, *pk, *pv,
            KV_F16 if dtype == torch.float16 else KV_F32, S, W, tokens, stream=stream)
    return outs[0], outs[1]


def cache8_copy_pages(cache: Cache8, src, dst, stream=None):
    """Copies page src[i] (codes and scales) to page dst[i] (int32 [n] each)."""
    dev = _cache8(cache).device
    ps, pd = _ints(src, "src", dev, 1), _ints(dst, "dst", dev, 1)
    if src.shape != dst.shape:
        raise ValueError("src and dst differ in length")
    _launch(cfp32_cache8_copy_pages, "cfp32_cache8_copy_pages", dev, cache.addr, ps, pd, src.shape[0], stream=stream)


def cache8_fork(cache: Cache8, table, lens, refs, parents, missing=None, refs_out=None,
                workspace: Workspace | None = None, stream=None):
    """``cache_fork`` of an 8-bit cache: (table, refs, lens) of the children."""
    torch = _torch()
    P, dev = _cache8(cache).shape[0], cache.device
    pt, pl, pr, pp = (_ints(table, "table", dev, 2), _ints(lens, "lens", dev, 1), _ints(refs, "refs", dev, 1),
                      _ints(parents, "parents", dev, 1))
    (S, W), C = table.shape, parents.shape[0]
    if lens.shape[0] != S or refs.shape[0] != P:
        raise ValueError("lens must have one entry per sequence, refs one per page")
    with torch.cuda.device(dev):
        table_out = _empty((C, W), torch.int32, dev, stream)
        lens_out = _empty(C, torch.int32, dev, stream)
        refs_out = _empty(refs.shape, torch.int32, dev, stream) if refs_out is None else refs_out
        pro = _ints(refs_out, "refs_out", dev, 1)
        pm = None if missing is None else _ints(missing, "missing", dev, 1)
        if refs_out.shape != refs.shape or (missing is not None and not missing.numel()):
            raise ValueError("refs_out or missing has the wrong shape")
        need = cfp32_cache_fork_workspace_bytes(C)
        buf, ws, st = _scratch(need, dev, workspace, stream)
        _check(cfp32_cache8_fork(cache.addr, pt, _ld(table), pl, pr, pp, table_out.data_ptr(), W, lens_out.data_ptr(), pro, pm,
                                 S, W, C, ws, need, st), "cfp32_cache8_fork")
    return table_out, refs_out, lens_out


def cache8_compact(cache: Cache8, table, refs, table_out=None, refs_out=None, workspace: Workspace | None = None,
                   stream=None):
    """``cache_compact`` of an 8-bit cache: (table, refs, n)."""
    torch = _torch()
    P, dev = _cache8(cache).shape[0], cache.device
    pt, pr = _ints(table, "table", dev, 2), _ints(refs, "refs", dev, 1)
    S, W = table.shape
    if refs.shape[0] != P:
        raise ValueError("refs must have one entry per page")
    with torch.cuda.device(dev):
        table_out = _empty((S, W), torch.int32, dev, stream) if table_out is None else table_out
        refs_out = _empty(refs.shape, torch.int32, dev, stream) if refs_out is None else refs_out
        pto, pro = _ints(table_out, "table_out", dev, 2), _ints(refs_out, "refs_out", dev, 1)
        if table_out.shape != table.shape or refs_out.shape != refs.shape:
            raise ValueError("table_out or refs_out has the wrong shape")
        live = _empty(1, torch.int32, dev, stream)
        need = cfp32_cache_compact_workspace_bytes(P)
        buf, ws, st = _scratch(need, dev, workspace, stream)
        _check(cfp32_cache8_compact(cache.addr, pt, _ld(table), pr, pto, _ld(table_out, "table_out"), pro, live.data_ptr(), S, W, ws, need,
                                    st), "cfp32_cache8_compact")
    return table_out, refs_out, live


def attention8_decode(q, cache: Cache8, table, lens, scale: float | None = None, out=None,
                      workspace: Workspace | None = None, stream=None):
    """Attention of one new token per sequence against an 8-bit cache: q FP32
    [B, Hq, D]; table int32 [B, W] (one row for all: ``row.expand(B, W)``);
    lens int32 [B].  Returns FP32 [B, Hq, D]."""
    torch = _torch()
    P, Hkv, page, D2 = _cache8(cache).shape
    if stream is None and workspace is None:
        done = _native().attention8_decode(q, cache.addr, cache.index, table, lens, scale, out)
        if done is not None:
            return done
    dev = cache.device
    pq = _heads(q, (torch.float32,), "q", dev)
    B, Hq, D = q.shape
    if D2 != D or Hkv == 0 or Hq % Hkv:
        raise ValueError("q and the pools differ in head size or heads")
    pt, pl = _ints(table, "table", dev, 2), _ints(lens, "lens", dev, 1)
    W = table.shape[1]
    if table.shape[0] != B or lens.shape[0] != B:
        raise ValueError("table and lens must have one row per sequence")
    with torch.cuda.device(dev):
        if out is None:
            out = _empty((B, Hq, D), torch.float32, dev, stream)
        elif out.shape != q.shape:
            raise ValueError("out has the wrong shape")
        po = _heads(out, (torch.float32,), "out", dev)
        need = cfp32_attention8_decode_workspace_bytes(B, Hq, Hkv, D, W, page)
        buf, ws, st = _scratch(need, dev, workspace, stream)
        _check(cfp32_attention8_decode(*pq, cache.addr, pt, _ld(table, shared=True), W, pl, *po, B, Hq,
                                       D ** -0.5 if scale is None else scale, ws, need, st), "cfp32_attention8_decode")
    return out


# -- beam search -----------------------------------------------------------------------

def beam_select(logits, scores, n: int | None = None, done=None, eos: int = -1, workspace: Workspace | None = None,
                stream=None):
    """(parents, tokens, scores, done), [S, n] each (n: as many beams as there
    are unless given; at most 64): the best continuations of S sequences.
    logits FP32 [S * beams, V], one row for all beams among them
    (``row.expand(S * beams, V)``); scores FP32 [S, beams], the beams' sums of
    log-probabilities; done bool [S, beams] or None; eos: the token that
    finishes a beam.  parents are rows of the batch of S * beams beams, as
    ``beam_reorder`` and ``cache_fork`` take them (-1 where there is no
    offer)."""
    if stream is None and workspace is None:
        done_ = _native().beam_select(logits, scores, n, done, eos)
        if done_ is not None:
            return done_
    torch = _torch()
    px, rows, V, ld = _mat(logits, (torch.float32,), "logits", shared=True)
    dev = logits.device
    if not isinstance(scores, torch.Tensor) or scores.dtype != torch.float32 or scores.device != dev:
        raise TypeError("scores: expected a float32 tensor on logits' device")
    if scores.dim() != 2 or not scores.is_contiguous() or scores.numel() != rows:
        raise ValueError("scores must be contiguous [sequences, beams], a beam to each row of logits")
    S, beams = scores.shape
    if done is not None:
        if not isinstance(done, torch.Tensor) or done.dtype not in (torch.bool, torch.uint8) or done.device != dev:
            raise TypeError("done: expected a bool tensor on logits' device")
        if done.shape != scores.shape or not done.is_contiguous():
            raise ValueError("done must be contiguous, of the shape of scores")
    n = beams if n is None else n
    with torch.cuda.device(dev):
        parents, tokens = (_empty((S, n), torch.int32, dev, stream) for _ in range(2))
        out, ended = _empty((S, n), torch.float32, dev, stream), _empty((S, n), torch.bool, dev, stream)
        need = cfp32_beam_select_workspace_bytes(S, beams, V, n)
        buf, ws, st = _scratch(need, dev, workspace, stream)
        _check(cfp32_beam_select(px, ld, scores.data_ptr(), None if done is None else done.data_ptr(), S, beams, V, n, eos,
                                 parents.data_ptr(), tokens.data_ptr(), out.data_ptr(), ended.data_ptr(), ws, need, st),
               "cfp32_beam_select")
    return parents, tokens, out, ended


def beam_reorder(states, parents, out=None, stream=None):
    """Rows of ``states`` [rows, ...] (any type, contiguous rows) in the order of
    ``parents`` (int32, any shape): [parents.numel(), ...]; zeros where a parent
    is no row."""
    if stream is None and out is None:
        done = _native().beam_reorder(states, parents)
        if done is not None:
            return done
    torch = _torch()
    if not isinstance(states, torch.Tensor) or states.device.type != "cuda":
        raise TypeError("states: expected a GPU tensor")
    dev = states.device
    if not isinstance(parents, torch.Tensor) or parents.dtype != torch.int32 or parents.device != dev:
        raise TypeError("parents: expected an int32 tensor on states' device")
    if not parents.is_contiguous():
        raise ValueError("parents must be contiguous")
    for t, name in ((states, "states"), (out, "out")):
        if t is not None and (t.is_conj() or t.is_neg()):
            raise ValueError(f"{name}: a view whose values are not those in memory (resolve_conj() or resolve_neg() copies it)")
    rest = states.shape[1:]
    if states.dim() < 1 or (states.shape[0] and not states[0].is_contiguous()):
        raise ValueError("states must have contiguous rows")
    shape, size = (parents.numel(), *rest), states.element_size()
    row = size
    for d in rest:
        row *= d
    if out is None:
        out = _empty(shape, states.dtype, dev, stream)
    elif out.shape != shape or out.dtype != states.dtype or out.device != dev or (shape[0] and not out[0].is_contiguous()):
        raise ValueError("out must have a row for each parent, of the type of states")

    def stride(t):
        return t.stride(0) * size if t.shape[0] > 1 else row

    _launch(cfp32_beam_reorder, "cfp32_beam_reorder", dev, states.data_ptr(), stride(states), out.data_ptr(), stride(out),
            parents.data_ptr(), states.shape[0], shape[0], row, stream=stream)
    return out
