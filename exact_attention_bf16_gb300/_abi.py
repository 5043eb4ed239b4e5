"""ctypes view of include/attn.h: the shared library, its status codes and the
parameter structs. Loading fails loudly if the library is missing; there is
no fallback implementation."""
from __future__ import annotations

import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libattn_gb300.so")
HEADER_PATH = os.path.join(os.path.dirname(HERE), "include", "attn.h")

ABI_VERSION = 9
BWD_NOALLOC_SCRATCH_BYTES = 8 << 20  # ATTN_BWD_NOALLOC_SCRATCH_BYTES

STATUS = {
    0: "ATTN_OK",
    1: "ATTN_ERR_INVALID_ARG",
    2: "ATTN_ERR_UNSUPPORTED",
    3: "ATTN_ERR_CUDA",
    4: "ATTN_ERR_TIMEOUT",
    5: "ATTN_ERR_WORKSPACE",
}
ATTN_OK, ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED, ATTN_ERR_CUDA, ATTN_ERR_TIMEOUT, ATTN_ERR_WORKSPACE = range(6)
SCORE_NONE, SCORE_SOFTCAP, SCORE_ALIBI, SCORE_RELBIAS = range(4)  # attn_score_mod_t
TABLE_BF16, TABLE_F32 = range(2)  # attn_table_dtype_t
INPUT_BF16, INPUT_E4M3 = range(2)  # attn_input_dtype_t

c_i32, c_i64, c_f32, c_vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


_REL_BIAS = [("rel_bias", c_vp), ("rel_bias_dtype", c_i32), ("rel_buckets", c_i32), ("rel_max_distance", c_i32),
             ("rel_bidirectional", c_i32)]


class AttnFwdParams(ctypes.Structure):
    _fields_ = [
        ("q", c_vp), ("k", c_vp), ("v", c_vp), ("o", c_vp), ("lse", c_vp),
        ("q_batch_stride", c_i64), ("q_row_stride", c_i64), ("q_head_stride", c_i64),
        ("k_batch_stride", c_i64), ("k_row_stride", c_i64), ("k_head_stride", c_i64),
        ("v_batch_stride", c_i64), ("v_row_stride", c_i64), ("v_head_stride", c_i64),
        ("o_batch_stride", c_i64), ("o_row_stride", c_i64), ("o_head_stride", c_i64),
        ("batch", c_i32), ("heads", c_i32), ("seqlen_q", c_i32), ("seqlen_k", c_i32),
        ("d_qk", c_i32), ("d_v", c_i32),
        ("cu_seqlens_q", c_vp), ("cu_seqlens_k", c_vp),
        ("num_seqs", c_i32), ("max_seqlen_q", c_i32), ("max_seqlen_k", c_i32),
        ("total_q", c_i32), ("total_k", c_i32),
        ("softmax_scale", c_f32), ("causal", c_i32), ("exp2_emu_period", c_i32),
        ("rescale_stats", c_vp),
        ("score_mod", c_i32), ("softcap", ctypes.c_float), ("alibi_slopes", c_vp),
        ("input_dtype", c_i32), ("q_descale", ctypes.c_float), ("k_descale", ctypes.c_float),
        ("v_descale", ctypes.c_float), ("cta_pair", c_i32), ("heads_kv", c_i32),
    ] + _REL_BIAS


class AttnBwdParams(ctypes.Structure):
    _fields_ = [
        ("fwd", AttnFwdParams),
        ("dout", c_vp), ("dq", c_vp), ("dk", c_vp), ("dv", c_vp),
        ("do_batch_stride", c_i64), ("do_row_stride", c_i64), ("do_head_stride", c_i64),
        ("dq_batch_stride", c_i64), ("dq_row_stride", c_i64), ("dq_head_stride", c_i64),
        ("dk_batch_stride", c_i64), ("dk_row_stride", c_i64), ("dk_head_stride", c_i64),
        ("dv_batch_stride", c_i64), ("dv_row_stride", c_i64), ("dv_head_stride", c_i64),
        ("deterministic", c_i32), ("cta_pair", c_i32),
        ("phase_events", c_vp * 3),
        ("single_pass", c_i32), ("drel_bias", c_vp),
    ]


class AttnKvPlanParams(ctypes.Structure):
    _fields_ = [
        ("seqlens_old", c_vp), ("seqlens_new", c_vp), ("block_table", c_vp), ("block_table_stride", c_i64),
        ("free_pages", c_vp), ("free_count", c_vp), ("free_count_out", c_vp), ("cu_seqlens_q", c_vp),
        ("seqlens_k", c_vp), ("slot_mapping", c_vp), ("status", c_vp),
        ("num_seqs", c_i32), ("max_pages", c_i32), ("page_size", c_i32), ("free_capacity", c_i32),
        ("max_tokens", c_i32), ("positions", c_vp),
    ]


class AttnKvAppendParams(ctypes.Structure):
    _fields_ = [
        ("k", c_vp), ("v", c_vp), ("k_cache", c_vp), ("v_cache", c_vp),
        ("k_row_stride", c_i64), ("k_head_stride", c_i64), ("v_row_stride", c_i64), ("v_head_stride", c_i64),
        ("k_cache_page_stride", c_i64), ("k_cache_row_stride", c_i64), ("k_cache_head_stride", c_i64),
        ("v_cache_page_stride", c_i64), ("v_cache_row_stride", c_i64), ("v_cache_head_stride", c_i64),
        ("slot_mapping", c_vp),
        ("tokens", c_i32), ("heads_kv", c_i32), ("d_qk", c_i32), ("d_v", c_i32), ("page_size", c_i32),
        ("num_pages", c_i32),
    ]


class AttnPagedParams(ctypes.Structure):
    _fields_ = [
        ("q", c_vp), ("k_cache", c_vp), ("v_cache", c_vp), ("o", c_vp), ("lse", c_vp),
        ("q_row_stride", c_i64), ("q_head_stride", c_i64), ("o_row_stride", c_i64), ("o_head_stride", c_i64),
        ("k_page_stride", c_i64), ("k_row_stride", c_i64), ("k_head_stride", c_i64),
        ("v_page_stride", c_i64), ("v_row_stride", c_i64), ("v_head_stride", c_i64),
        ("block_table", c_vp), ("block_table_stride", c_i64), ("cu_seqlens_q", c_vp), ("seqlens_k", c_vp),
        ("num_seqs", c_i32), ("heads", c_i32), ("heads_kv", c_i32), ("d_qk", c_i32), ("d_v", c_i32),
        ("page_size", c_i32), ("num_pages", c_i32), ("max_pages", c_i32), ("total_q", c_i32), ("max_seqlen_q", c_i32),
        ("softmax_scale", c_f32), ("causal", c_i32), ("score_mod", c_i32), ("softcap", c_f32), ("alibi_slopes", c_vp),
    ] + _REL_BIAS


class AttnRotaryParams(ctypes.Structure):
    _fields_ = [
        ("q", c_vp), ("k", c_vp), ("q_out", c_vp), ("k_out", c_vp),
        ("q_batch_stride", c_i64), ("q_row_stride", c_i64), ("q_head_stride", c_i64),
        ("k_batch_stride", c_i64), ("k_row_stride", c_i64), ("k_head_stride", c_i64),
        ("q_out_batch_stride", c_i64), ("q_out_row_stride", c_i64), ("q_out_head_stride", c_i64),
        ("k_out_batch_stride", c_i64), ("k_out_row_stride", c_i64), ("k_out_head_stride", c_i64),
        ("positions", c_vp), ("positions_batch_stride", c_i64),
        ("cos_table", c_vp), ("sin_table", c_vp), ("table_row_stride", c_i64),
        ("batch", c_i32), ("seqlen", c_i32), ("heads", c_i32), ("heads_kv", c_i32), ("d_qk", c_i32),
        ("rotary_dim", c_i32), ("rotary_offset", c_i32), ("interleaved", c_i32), ("inverse", c_i32),
        ("num_positions", c_i32),
    ]


class AttnKvAppendRotaryParams(ctypes.Structure):
    _fields_ = [
        ("append", AttnKvAppendParams),
        ("q", c_vp), ("q_out", c_vp),
        ("q_row_stride", c_i64), ("q_head_stride", c_i64), ("q_out_row_stride", c_i64), ("q_out_head_stride", c_i64),
        ("positions", c_vp), ("cos_table", c_vp), ("sin_table", c_vp), ("table_row_stride", c_i64),
        ("heads", c_i32), ("rotary_dim", c_i32), ("rotary_offset", c_i32), ("interleaved", c_i32),
        ("num_positions", c_i32),
    ]


_CODES = {c_i32: "i", c_i64: "q", c_f32: "f", c_vp: "P"}


def _format(cls) -> str:
    out = ""
    for _, t in cls._fields_:
        if t in _CODES:
            out += _CODES[t]
        elif issubclass(t, ctypes.Array):
            out += _CODES[t._type_] * t._length_
        else:
            out += _format(t)
    return out


def packer(cls):
    """A function from a parameter struct's fields (in order, nested ones flattened, pointers as ints) to its bytes,
    which the entry points take in its place: one call instead of an attribute set per field."""
    s = struct.Struct("@" + _format(cls) + "0P")
    if s.size != ctypes.sizeof(cls):
        raise ImportError(f"{cls.__name__}: packed size {s.size} != {ctypes.sizeof(cls)}")
    return s.pack


_lib = None


def load(path: str = LIB_PATH):
    """Loads libattn_gb300.so and declares the C signatures (once)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python exact_attention_bf16_gb300/build.py` "
            "(nvcc, sm_103a). There is no non-CUDA fallback.")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    # parameter structs: byref(struct) or its packed bytes
    sig = {
        "attn_fwd_workspace_size": (ctypes.c_size_t, [c_vp]),
        "attn_bwd_workspace_size": (ctypes.c_size_t, [c_vp]),
        "attn_fwd_varlen_workspace_size": (ctypes.c_size_t, [c_vp]),
        "attn_bwd_varlen_workspace_size": (ctypes.c_size_t, [c_vp]),
        "attn_fwd": (ctypes.c_int, [c_vp, c_vp, ctypes.c_size_t, c_vp]),
        "attn_fwd_varlen": (ctypes.c_int, [c_vp, c_vp, ctypes.c_size_t, c_vp]),
        "attn_fwd_block_sparse": (ctypes.c_int, [c_vp, c_vp, c_vp, ctypes.c_int32, ctypes.c_int32, c_vp,
                                                 ctypes.c_size_t, c_vp]),
        "attn_bwd_block_sparse_workspace_size": (ctypes.c_size_t, [c_vp, ctypes.c_int32]),
        "attn_bwd_block_sparse": (ctypes.c_int, [c_vp, c_vp, c_vp, ctypes.c_int32, ctypes.c_int32, c_vp,
                                                 ctypes.c_size_t, c_vp]),
        "attn_bwd": (ctypes.c_int, [c_vp, c_vp, ctypes.c_size_t, c_vp]),
        "attn_bwd_varlen": (ctypes.c_int, [c_vp, c_vp, ctypes.c_size_t, c_vp]),
        "attn_bwd_noalloc": (ctypes.c_int, [c_vp, c_vp]),
        "attn_kv_plan": (ctypes.c_int, [c_vp, c_vp]),
        "attn_kv_append": (ctypes.c_int, [c_vp, c_vp]),
        "attn_rotary": (ctypes.c_int, [c_vp, c_vp]),
        "attn_kv_append_rotary": (ctypes.c_int, [c_vp, c_vp]),
        "attn_fwd_paged_workspace_size": (ctypes.c_size_t, [c_vp]),
        "attn_fwd_paged": (ctypes.c_int, [c_vp, c_vp, ctypes.c_size_t, c_vp]),
        "attn_kv_plan_params_size": (ctypes.c_size_t, []),
        "attn_kv_append_params_size": (ctypes.c_size_t, []),
        "attn_paged_params_size": (ctypes.c_size_t, []),
        "attn_rotary_params_size": (ctypes.c_size_t, []),
        "attn_kv_append_rotary_params_size": (ctypes.c_size_t, []),
        "attn_exp2_eval": (ctypes.c_int, [c_vp, c_vp, c_vp, c_i64, c_vp]),
        "attn_diag_wait_timeout": (ctypes.c_int, [c_vp, ctypes.c_uint32, c_vp]),
        "attn_get_device_status": (ctypes.c_int, [c_vp, P(ctypes.c_uint32)]),
        "attn_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "attn_last_cuda_error": (ctypes.c_char_p, []),
        "attn_abi_version": (c_i32, []),
        "attn_fwd_params_size": (ctypes.c_size_t, []),
        "attn_bwd_params_size": (ctypes.c_size_t, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if lib.attn_abi_version() != ABI_VERSION:
        raise ImportError(f"libattn_gb300.so ABI {lib.attn_abi_version()} != binding ABI {ABI_VERSION}")
    if lib.attn_fwd_params_size() != ctypes.sizeof(AttnFwdParams) or \
            lib.attn_bwd_params_size() != ctypes.sizeof(AttnBwdParams) or \
            lib.attn_kv_plan_params_size() != ctypes.sizeof(AttnKvPlanParams) or \
            lib.attn_kv_append_params_size() != ctypes.sizeof(AttnKvAppendParams) or \
            lib.attn_paged_params_size() != ctypes.sizeof(AttnPagedParams) or \
            lib.attn_rotary_params_size() != ctypes.sizeof(AttnRotaryParams) or \
            lib.attn_kv_append_rotary_params_size() != ctypes.sizeof(AttnKvAppendRotaryParams):
        raise ImportError("libattn_gb300.so parameter-struct layout differs from the binding")
    _lib = lib
    return lib


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = _lib
        detail = lib.attn_last_cuda_error().decode() if (lib is not None and status == ATTN_ERR_CUDA) else ""
        super().__init__(f"{where}: {STATUS.get(status, status)}" + (f" ({detail})" if detail else ""))
        self.status = status


def check(status: int, where: str):
    if status != ATTN_OK:
        raise AttnError(status, where)
