"""Exact fused scaled-dot-product attention (bf16) for NVIDIA GB300 (sm_103a).

The compute lives in libattn_gb300.so (hand-written CUDA: TMA, tcgen05 MMAs
with Tensor Memory accumulators, warp-specialised pipelines); see
include/attn.h for the C ABI. This package is a thin binding with the same
entry-point names: it only marshals torch tensors (device memory, strides,
the current CUDA stream) into the C parameter structs. Nothing here computes
attention, and there is no CPU or library fallback: if the shared library is
missing, importing this package raises.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple, Union

import torch

from . import _abi
from ._abi import (AttnBwdParams, AttnError, AttnFwdParams, AttnKvAppendParams, AttnKvAppendRotaryParams,  # noqa: F401
                   AttnKvPlanParams, AttnPagedParams, AttnRotaryParams)

_lib = _abi.load()

SUPPORTED_HEAD_DIMS = ((64, 64), (128, 128), (192, 128))

__all__ = [
    "attn_fwd", "attn_fwd_block_sparse", "attn_fwd_varlen", "attn_bwd", "attn_bwd_block_sparse",
    "block_lists_from_mask", "attn_bwd_varlen", "attn_exp2_eval",
    "attn_kv_plan", "attn_kv_append", "attn_kv_append_rotary", "attn_fwd_paged", "attn_rotary", "attn_get_device_status",
    "attention", "attention_varlen", "rotary", "AttnError", "SUPPORTED_HEAD_DIMS", "library_path",
]


def library_path() -> str:
    return _abi.LIB_PATH


_BF16, _I32, _I64, _F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
_pack_fwd, _pack_bwd = _abi.packer(AttnFwdParams), _abi.packer(AttnBwdParams)
_pack_plan, _pack_append, _pack_paged = (_abi.packer(AttnKvPlanParams), _abi.packer(AttnKvAppendParams),
                                         _abi.packer(AttnPagedParams))
_pack_rotary, _pack_append_rotary = _abi.packer(AttnRotaryParams), _abi.packer(AttnKvAppendRotaryParams)
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream_of(stream, t: torch.Tensor) -> int:
    """The stream handle of a call on t's GPU: the given one, or the current one of that GPU."""
    if stream is None:
        return _raw_stream(t.get_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _bf16_layout(name: str, t, ndim: int):
    """(shape, strides) of a checked bf16 CUDA tensor with contiguous last dim; a dim of at most one element, whose
    stride may be anything, gets a valid one."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _BF16 or not t.is_cuda or t.dim() != ndim:
        _check_bf16(name, t, ndim)
    shape, stride = t.shape, t.stride()
    if stride[-1] != 1:
        _check_bf16(name, t, ndim)
    if 1 in shape:
        stride = tuple(s if n > 1 else shape[-1] for s, n in zip(stride, shape))
    return shape, stride


_NO_REL = (0, 0, 0, 0, 0)


def _mod_fields(q, softcap, alibi_slopes, rel_bias=None, rel_max_distance=128, rel_bidirectional=True):
    """(score_mod, softcap, alibi_slopes) and the bias's fields (rel_bias .. rel_bidirectional) of a call (attn_fwd)."""
    if softcap is None and alibi_slopes is None:
        if rel_bias is None:
            return (0, 0.0, 0), _NO_REL
        return (_abi.SCORE_RELBIAS, 0.0, 0), _rel_fields(q, rel_bias, rel_max_distance, rel_bidirectional)
    p = AttnFwdParams()
    _set_score_mod(p, q, softcap, alibi_slopes, rel_bias)
    return (p.score_mod, p.softcap, p.alibi_slopes or 0), _NO_REL


def _rel_fields(q, t, rel_max_distance, rel_bidirectional):
    """rel_bias .. rel_bidirectional of a checked table."""
    if not isinstance(t, torch.Tensor) or t.dtype not in (_BF16, _F32) or not t.is_cuda or not t.is_contiguous() or \
            t.dim() != 2 or t.shape[1] != q.shape[-2]:
        raise ValueError(f"rel_bias must be a contiguous bfloat16 or float32 CUDA tensor [buckets, {q.shape[-2]}]")
    if t.get_device() != q.get_device():
        raise ValueError(f"rel_bias is on {t.device} but q is on {q.device}")
    if not 0 < rel_max_distance < 2 ** 31:
        raise ValueError(f"rel_max_distance {rel_max_distance} must be a positive 32-bit number")
    return (t.data_ptr(), _abi.TABLE_F32 if t.dtype is _F32 else _abi.TABLE_BF16, t.shape[0], int(rel_max_distance),
            1 if rel_bidirectional else 0)


def _check_int32(name: str, t, device: int, n: int):
    if not isinstance(t, torch.Tensor) or t.dtype is not _I32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device} but the call is on cuda:{device}")
    if t.dim() != 1 or (n >= 0 and t.shape[0] != n):
        raise ValueError(f"{name} must have shape ({n if n >= 0 else 'n'},), got {tuple(t.shape)}")


def _stream(stream, device=None) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _check_bf16(name: str, t: torch.Tensor, ndim: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if t.stride(-1) != 1:
        raise ValueError(f"{name}: head_dim must be contiguous")


def _check_inputs(q, k, v, ndim: int) -> bool:
    """q, k, v all bf16, or all FP8 E4M3 (torch.float8_e4m3fn, forward only); returns True for E4M3."""
    f8 = q.dtype == torch.float8_e4m3fn
    for n, t in (("q", q), ("k", k), ("v", v)):
        if f8:
            if not isinstance(t, torch.Tensor) or t.dtype != torch.float8_e4m3fn:
                raise TypeError(f"{n} must be float8_e4m3fn like q")
            if not t.is_cuda or t.dim() != ndim or t.stride(-1) != 1:
                raise ValueError(f"{n} must be a CUDA tensor of {ndim} dims with contiguous head_dim")
        else:
            _check_bf16(n, t, ndim)
    return f8


def _set_input_dtype(p: AttnFwdParams, f8: bool, q_descale, k_descale, v_descale):
    if f8:
        p.input_dtype = _abi.INPUT_E4M3
        p.q_descale, p.k_descale, p.v_descale = float(q_descale), float(k_descale), float(v_descale)


def _strides4(t: torch.Tensor):
    # [B, N, H, d] -> (batch, row, head) element strides
    return t.stride(0), t.stride(1), t.stride(2)


def _strides3(t: torch.Tensor):
    # packed [total, H, d] -> batch stride unused
    return 0, t.stride(0), t.stride(1)


def _fill_fwd(p: AttnFwdParams, q, k, v, o, lse, strides, scale, causal):
    p.q, p.k, p.v, p.o, p.lse = _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse)
    (p.q_batch_stride, p.q_row_stride, p.q_head_stride) = strides(q)
    (p.k_batch_stride, p.k_row_stride, p.k_head_stride) = strides(k)
    (p.v_batch_stride, p.v_row_stride, p.v_head_stride) = strides(v)
    (p.o_batch_stride, p.o_row_stride, p.o_head_stride) = strides(o)
    p.d_qk, p.d_v = q.shape[-1], v.shape[-1]
    p.heads, p.heads_kv = q.shape[-2], k.shape[-2]
    p.softmax_scale = scale
    p.causal = 1 if causal else 0


def _set_score_mod(p: AttnFwdParams, q: torch.Tensor, softcap, alibi_slopes, rel_bias=None, rel_max_distance=128,
                   rel_bidirectional=True):
    """Score modification: logits soft-capped at ``softcap`` (a' = c tanh(a / c)), or ALiBi with one
    slope per head (``alibi_slopes`` float32 [H] on q's GPU, each >= 0), or a learned bias by buckets of relative
    position (``rel_bias`` [buckets, H], bf16 or float32, on q's GPU)."""
    if (softcap is not None) + (alibi_slopes is not None) + (rel_bias is not None) > 1:
        raise ValueError("choose one score modification: softcap, alibi_slopes or rel_bias")
    if rel_bias is not None:
        p.score_mod = _abi.SCORE_RELBIAS
        (p.rel_bias, p.rel_bias_dtype, p.rel_buckets, p.rel_max_distance, p.rel_bidirectional) = _rel_fields(
            q, rel_bias, rel_max_distance, rel_bidirectional)
    elif softcap is not None:
        p.score_mod, p.softcap = _abi.SCORE_SOFTCAP, float(softcap)
    elif alibi_slopes is not None:
        t = alibi_slopes
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous() or t.shape != (q.shape[-2],):
            raise ValueError(f"alibi_slopes must be a contiguous float32 CUDA tensor of shape [{q.shape[-2]}]")
        if t.device != q.device:
            raise ValueError(f"alibi_slopes is on {t.device} but q is on {q.device}")
        p.score_mod, p.alibi_slopes = _abi.SCORE_ALIBI, _ptr(t)


def _workspace(size: int, device, stream=None) -> Tuple[Optional[torch.Tensor], int]:
    if size == 0:
        return None, 0
    ws = torch.empty(size, dtype=torch.uint8, device=device)
    _used_on(stream, ws)
    return ws, size


def _workspace_ptr(size: int, like: torch.Tensor, stream):
    """(the tensor, which must live until the call has been made; its address)"""
    if size == 0:
        return None, 0
    ws = torch.empty(size, dtype=torch.uint8, device=like.device)
    if stream is not None:
        _used_on(stream, ws)
    return ws, ws.data_ptr()


def _used_on(stream, *tensors):
    """Tensors that a call allocates belong to the current stream; when the call runs on another one,
    their memory must not be handed out again before that stream is done with it."""
    if stream is None:
        return
    for t in tensors:
        s = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=t.device)
        if s.cuda_stream != torch.cuda.current_stream(t.device).cuda_stream:
            t.record_stream(s)


def _check_offsets(q, cu_seqlens_q, cu_seqlens_k):
    """The packed sequences' offsets: int32 [sequences + 1] on q's GPU, as many of q as of k."""
    dev = q.get_device()
    _check_int32("cu_seqlens_q", cu_seqlens_q, dev, -1)
    if cu_seqlens_k is not cu_seqlens_q:
        _check_int32("cu_seqlens_k", cu_seqlens_k, dev, cu_seqlens_q.shape[0])


def _check_packed_kv(q, k, v, heads: int, d_qk: int, ks, vs) -> int:
    """Packed k [total_k, Hkv, d_qk] and v [total_k, Hkv, d_v] against q's heads, Hkv a divisor of them; q's GPU."""
    if ks[2] != d_qk or ks[0] != vs[0] or ks[1] != vs[1] or ks[1] < 1 or heads % ks[1] != 0:
        _check_kv(q, k, v)
    dev = q.get_device()
    if k.get_device() != dev or v.get_device() != dev:
        _check_kv(q, k, v)
    return dev


def _packed_grad(name: str, grad, like, stream):
    """A gradient buffer for `like` (the given one, checked) and its strides."""
    if grad is None:
        grad = torch.empty(like.shape, dtype=_BF16, device=like.device) if like.is_contiguous() else torch.empty_like(like)
        if stream is not None:
            _used_on(stream, grad)
    elif grad.shape != like.shape or grad.device != like.device:
        raise ValueError(f"{name} must be {tuple(like.shape)} on {like.device}, got {tuple(grad.shape)} on {grad.device}")
    return grad, _bf16_layout(name, grad, 3)[1]


def _check_kv(q, k, v):
    """k and v of a call whose query heads may share K/V heads: q [..., H, d_qk], k [..., Hkv, d_qk] and
    v [..., Hkv, d_v] with Hkv a divisor of H, rows of k and v alike (dense: batches of q alike)."""
    h, hk = q.shape[-2], k.shape[-2]
    if k.shape[-1] != q.shape[-1] or v.shape[:-1] != k.shape[:-1] or (k.dim() == 4 and k.shape[0] != q.shape[0]):
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)}")
    if hk < 1 or h % hk != 0:
        raise ValueError(f"{hk} K/V heads do not divide {h} query heads")
    dev = q.get_device()
    for n, t in (("k", k), ("v", v)):
        if t.get_device() != dev:
            raise ValueError(f"{n} is on {t.device} but q is on {q.device}")


def _check_bwd(q, k, v, out, lse, dout, lse_shape, grads):
    """The forward's outputs and dO of a backward call, and gradient buffers the caller passed in."""
    _check_kv(q, k, v)
    want = q.shape[:-1] + v.shape[-1:]
    for n, t in (("out", out), ("dout", dout)):
        if t.shape != want:
            raise ValueError(f"{n} must be {tuple(want)}, got {tuple(t.shape)}")
    if tuple(lse.shape) != lse_shape or not lse.is_contiguous() or lse.dtype != torch.float32:
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {lse_shape}")
    for n, t, like in (("dq", grads[0], q), ("dk", grads[1], k), ("dv", grads[2], v)):
        if t is not None:
            _check_bf16(n, t, like.dim())
            if t.shape != like.shape:
                raise ValueError(f"{n} must be {tuple(like.shape)}, got {tuple(t.shape)}")
    dev = q.get_device()
    for n, t in (("out", out), ("lse", lse), ("dout", dout)):
        if t.get_device() != dev:
            raise ValueError(f"{n} is on {t.device} but q is on {q.device}")


def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, causal: bool = False,
             softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
             lse: Optional[torch.Tensor] = None, rescale_stats: Optional[torch.Tensor] = None,
             exp2_emu_period: int = 0, softcap: Optional[float] = None,
             alibi_slopes: Optional[torch.Tensor] = None, q_descale: float = 1.0, k_descale: float = 1.0,
             v_descale: float = 1.0, cta_pair: bool = False, rel_bias: Optional[torch.Tensor] = None, rel_max_distance: int = 128,
             rel_bidirectional: bool = True, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Dense forward. q [B, Nq, H, d_qk], k [B, Nk, Hkv, d_qk], v [B, Nk, Hkv, d_v] (bf16, CUDA); Hkv
    divides H, and query head h reads K/V head h // (H // Hkv).
    Returns (O [B, Nq, H, d_v] bf16, LSE [B, H, Nq] fp32, natural log). ``exp2_emu_period`` (0, 4, 8)
    sends one column in that many of every row's exp2 to the FMA-pipe polynomial. ``softcap``,
    ``alibi_slopes`` or ``rel_bias`` select a score modification (include/attn.h, attn_fwd_params.score_mod):
    ``rel_bias`` [buckets, H] (bf16 or float32, up to 128 buckets) adds a learned bias by the bucket of the key's position
    relative to the query's, both sides apart with ``rel_bidirectional`` (else all keys behind the query share bucket 0),
    whole distances first and then logarithmic up to ``rel_max_distance`` (attn_fwd_params.rel_bias); -inf masks a bucket, and
    finite entries count up to +-65536.
    q, k, v may instead all be torch.float8_e4m3fn (d = 128), standing for their values times
    ``q_descale``, ``k_descale``, ``v_descale``. ``cta_pair`` runs the two-SM forward (d = 128)."""
    f8 = _check_inputs(q, k, v, 4)
    B, Nq, H, dqk = q.shape
    Nk, dv = k.shape[1], v.shape[-1]
    _check_kv(q, k, v)
    scale = float(softmax_scale) if softmax_scale is not None else 1.0 / math.sqrt(dqk)
    if out is None:
        out = torch.empty((B, Nq, H, dv), dtype=torch.bfloat16, device=q.device)
        _used_on(stream, out)
    _check_bf16("out", out, 4)
    if out.shape != (B, Nq, H, dv):
        raise ValueError(f"out must be {(B, Nq, H, dv)}, got {tuple(out.shape)}")
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
        _used_on(stream, lse)
    if (lse.shape != (B, H, Nq) or not lse.is_contiguous() or lse.dtype != torch.float32 or lse.device != q.device or
            out.device != q.device):
        raise ValueError(f"out and lse (a contiguous float32 [B, H, Nq] tensor) must be on {q.device}")
    p = AttnFwdParams()
    _fill_fwd(p, q, k, v, out, lse, _strides4, scale, causal)
    p.batch, p.seqlen_q, p.seqlen_k = B, Nq, Nk
    p.rescale_stats = _ptr(rescale_stats)
    p.exp2_emu_period = int(exp2_emu_period)
    _set_score_mod(p, q, softcap, alibi_slopes, rel_bias, rel_max_distance, rel_bidirectional)
    _set_input_dtype(p, f8, q_descale, k_descale, v_descale)
    p.cta_pair = 1 if cta_pair else 0
    ws, nbytes = _workspace(_lib.attn_fwd_workspace_size(ctypes.byref(p)), q.device, stream)
    _abi.check(_lib.attn_fwd(ctypes.byref(p), _ptr(ws), nbytes, _stream(stream, q.device)), "attn_fwd")
    return out, lse


def _check_lists(q: torch.Tensor, kv_count: torch.Tensor, kv_index: torch.Tensor) -> Tuple[int, int]:
    """Validates the block lists of a dense [B, Nq, H, d] call; returns (max_kv, lists_per_head).
    Shared lists: kv_count [nqb], kv_index [nqb, max_kv]. Per (batch, head): kv_count [B, H, nqb],
    kv_index [B, H, nqb, max_kv]."""
    for n, t in (("kv_count", kv_count), ("kv_index", kv_index)):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous int32 CUDA tensor")
        if t.device != q.device:
            raise ValueError(f"{n} is on {t.device} but q is on {q.device}: the block lists must be on q's GPU")
    B, Nq, H = q.shape[0], q.shape[1], q.shape[2]
    nqb = (Nq + 255) // 256
    if kv_count.shape == (nqb,) and kv_index.dim() == 2 and kv_index.shape[0] == nqb:
        return int(kv_index.shape[1]), 0
    if kv_count.shape == (B, H, nqb) and kv_index.dim() == 4 and kv_index.shape[:3] == (B, H, nqb):
        return int(kv_index.shape[3]), 1
    raise ValueError(f"kv_count must be [{nqb}] and kv_index [{nqb}, max_kv], or per (batch, head) "
                     f"[{B}, {H}, {nqb}] and [{B}, {H}, {nqb}, max_kv]")


def block_lists_from_mask(block_mask: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """(kv_count, kv_index) for :func:`attn_fwd_block_sparse` from a boolean block mask
    [ceil(Nq/256), ceil(Nk/128)], or [B, H, ceil(Nq/256), ceil(Nk/128)] for lists per (batch, head)
    (True = the query block attends to the key block), key blocks in ascending order; on the mask's
    device. Argument preparation only."""
    if block_mask.dtype != torch.bool or block_mask.dim() not in (2, 4):
        raise ValueError("block_mask must be a bool tensor [query blocks, key blocks] or [B, H, query blocks, "
                         "key blocks]")
    m = block_mask.to(torch.int32)
    kv_count = m.sum(dim=-1, dtype=torch.int32)
    max_kv = max(int(kv_count.max().item()) if kv_count.numel() else 0, 1)
    # stable sort puts listed blocks first, each group in ascending key-block order
    order = torch.sort(1 - m, dim=-1, stable=True).indices.to(torch.int32)
    kv_index = order[..., :max_kv].contiguous()
    return kv_count.contiguous(), kv_index


def attn_fwd_block_sparse(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_count: torch.Tensor,
                          kv_index: torch.Tensor, *, causal: bool = False, softmax_scale: Optional[float] = None,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          softcap: Optional[float] = None, alibi_slopes: Optional[torch.Tensor] = None,
                          stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Block-sparse dense forward. q/k/v as in :func:`attn_fwd`; kv_count int32 [ceil(Nq/256)] and
    kv_index int32 [ceil(Nq/256), max_kv] (CUDA, contiguous): query block b (rows 256b..256b+255)
    attends to key blocks (of 128 keys) kv_index[b, :kv_count[b]], each listed at most once; or per
    (batch, head), kv_count [B, H, nqb] and kv_index [B, H, nqb, max_kv].
    Returns (O [B, Nq, H, d_v] bf16, LSE [B, H, Nq] fp32)."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _check_bf16(n, t, 4)
    B, Nq, H, dqk = q.shape
    Nk, dv = k.shape[1], v.shape[-1]
    if k.shape != (B, Nk, H, dqk) or v.shape[:3] != (B, Nk, H):
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)}")
    max_kv, per_head = _check_lists(q, kv_count, kv_index)
    scale = float(softmax_scale) if softmax_scale is not None else 1.0 / math.sqrt(dqk)
    if out is None:
        out = torch.empty((B, Nq, H, dv), dtype=torch.bfloat16, device=q.device)
    _check_bf16("out", out, 4)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if (lse.shape != (B, H, Nq) or not lse.is_contiguous() or lse.dtype != torch.float32 or lse.device != q.device or
            out.device != q.device):
        raise ValueError(f"out and lse (a contiguous float32 [B, H, Nq] tensor) must be on {q.device}")
    p = AttnFwdParams()
    _fill_fwd(p, q, k, v, out, lse, _strides4, scale, causal)
    p.batch, p.seqlen_q, p.seqlen_k = B, Nq, Nk
    _set_score_mod(p, q, softcap, alibi_slopes)
    ws, nbytes = _workspace(_lib.attn_fwd_workspace_size(ctypes.byref(p)), q.device, stream)
    _abi.check(_lib.attn_fwd_block_sparse(ctypes.byref(p), _ptr(kv_count), _ptr(kv_index), max_kv, per_head,
                                          _ptr(ws), nbytes, _stream(stream, q.device)), "attn_fwd_block_sparse")
    return out, lse


def attn_fwd_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                    cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int, *, causal: bool = False,
                    softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, rescale_stats: Optional[torch.Tensor] = None,
                    exp2_emu_period: int = 0, softcap: Optional[float] = None,
                    alibi_slopes: Optional[torch.Tensor] = None, q_descale: float = 1.0, k_descale: float = 1.0,
                    v_descale: float = 1.0, cta_pair: bool = False, rel_bias: Optional[torch.Tensor] = None, rel_max_distance: int = 128,
                    rel_bidirectional: bool = True,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Packed variable-length forward. q [total_q, H, d_qk], k/v [total_k, Hkv, d] with Hkv a divisor of H
    (query head h reads K/V head h // (H // Hkv)); cu_seqlens int32 on the device. Sequences do not reach one another,
    whatever their rows, or spare rows behind the last offset, hold. Returns
    (O [total_q, H, d_v], LSE [H, total_q]). Score modifications and E4M3 inputs as in :func:`attn_fwd`,
    positions counted within each sequence."""
    f8 = q.dtype is torch.float8_e4m3fn
    if f8:
        _check_inputs(q, k, v, 3)
        (tq, H, dqk), sq, ks, sk, vs, sv = q.shape, q.stride(), k.shape, k.stride(), v.shape, v.stride()
    else:
        ((tq, H, dqk), sq), (ks, sk), (vs, sv) = (_bf16_layout("q", q, 3), _bf16_layout("k", k, 3),
                                                  _bf16_layout("v", v, 3))
    _check_offsets(q, cu_seqlens_q, cu_seqlens_k)
    _check_packed_kv(q, k, v, H, dqk, ks, vs)
    tk, dv = ks[0], vs[2]
    scale = float(softmax_scale) if softmax_scale is not None else 1.0 / math.sqrt(dqk)
    if out is None:
        out, so = torch.empty((tq, H, dv), dtype=_BF16, device=q.device), (H * dv, dv)
    else:
        shape, so = _bf16_layout("out", out, 3)
        if shape != (tq, H, dv) or out.device != q.device:
            raise ValueError(f"out must be {(tq, H, dv)} on {q.device}, got {tuple(shape)} on {out.device}")
    if lse is None:
        lse = torch.empty((H, tq), dtype=_F32, device=q.device)
    elif lse.shape != (H, tq) or not lse.is_contiguous() or lse.dtype is not _F32 or lse.device != q.device:
        raise ValueError(f"lse must be a contiguous float32 [H, total_q] tensor on {q.device}")
    if stream is not None:
        _used_on(stream, out, lse)
    mod, rel = _mod_fields(q, softcap, alibi_slopes, rel_bias, rel_max_distance, rel_bidirectional)
    p = _pack_fwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
        0, sq[0], sq[1], 0, sk[0], sk[1], 0, sv[0], sv[1], 0, so[0], so[1],
        1, H, 0, 0, dqk, dv, cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), cu_seqlens_q.shape[0] - 1,
        int(max_seqlen_q), int(max_seqlen_k), tq, tk, scale, 1 if causal else 0, int(exp2_emu_period),
        rescale_stats.data_ptr() if rescale_stats is not None else 0, *mod,
        _abi.INPUT_E4M3 if f8 else _abi.INPUT_BF16, float(q_descale), float(k_descale), float(v_descale),
        1 if cta_pair else 0, ks[1], *rel)
    nbytes = _lib.attn_fwd_varlen_workspace_size(p)
    ws, ws_ptr = _workspace_ptr(nbytes, q, stream)
    status = _lib.attn_fwd_varlen(p, ws_ptr, nbytes, _stream_of(stream, q))
    if status:
        _abi.check(status, "attn_fwd_varlen")
    return out, lse


def _fill_bwd(p: AttnBwdParams, do, dq, dk, dv, strides, deterministic, cta_pair=False, single_pass=False):
    p.dout, p.dq, p.dk, p.dv = _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv)
    (p.do_batch_stride, p.do_row_stride, p.do_head_stride) = strides(do)
    (p.dq_batch_stride, p.dq_row_stride, p.dq_head_stride) = strides(dq)
    (p.dk_batch_stride, p.dk_row_stride, p.dk_head_stride) = strides(dk)
    (p.dv_batch_stride, p.dv_row_stride, p.dv_head_stride) = strides(dv)
    p.deterministic = 1 if deterministic else 0
    p.cta_pair = 1 if cta_pair else 0
    p.single_pass = 1 if single_pass else 0


def _rel_grad(drel_bias, rel_bias, wanted: bool, stream):
    """The buffer for rel_bias's gradient (the given one, checked), or None."""
    if rel_bias is None or not wanted:
        if drel_bias is not None:
            raise ValueError("drel_bias without rel_bias, or without rel_bias_grad")
        return None
    if drel_bias is None:
        drel_bias = torch.empty_like(rel_bias)
        _used_on(stream, drel_bias)
    elif drel_bias.shape != rel_bias.shape or drel_bias.dtype is not rel_bias.dtype or drel_bias.device != rel_bias.device or \
            not drel_bias.is_contiguous():
        raise ValueError(f"drel_bias must be a contiguous {rel_bias.dtype} tensor {tuple(rel_bias.shape)} on {rel_bias.device}")
    return drel_bias


def _grad_buffers(stream, *pairs):
    out = []
    for grad, like in pairs:
        if grad is None:
            grad = torch.empty_like(like)
            _used_on(stream, grad)
        out.append(grad)
    return out


def _event_handles(events):
    if events is None:
        return None
    out = []
    for ev in events:
        if ev is None:
            out.append(None)
            continue
        if getattr(ev, "cuda_event", 0) == 0:  # torch creates the CUDA event lazily
            ev.record()
        out.append(ev.cuda_event)
    return out


def attn_bwd(q, k, v, out, lse, dout, *, causal: bool = False, softmax_scale: Optional[float] = None,
             deterministic: bool = False, dq=None, dk=None, dv=None, stream=None, phase_events=None,
             cta_pair: bool = False, softcap: Optional[float] = None, alibi_slopes: Optional[torch.Tensor] = None,
             single_pass: bool = False, rel_bias: Optional[torch.Tensor] = None, rel_max_distance: int = 128,
             rel_bidirectional: bool = True, drel_bias: Optional[torch.Tensor] = None, rel_bias_grad: bool = True):
    """Dense backward: returns (dQ, dK, dV) bf16 for the loss <O, dO>; where query heads share K/V heads
    (attn_fwd), dK and dV are the sums over them. ``phase_events`` (optional, three
    torch.cuda.Event) are recorded after the D pass, the dK/dV kernel and the dQ kernel. ``cta_pair``
    selects the two-SM (cta_group::2) dK/dV kernel (d = 128); ``single_pass`` the one-kernel backward
    whose dQ partials are reduced across CTAs (d = 64; ordered by key tile when ``deterministic``).
    The score modification must be the forward's. With ``rel_bias`` a fourth value is returned, its gradient in
    its type (into ``drel_bias`` when given; None, and not computed, without ``rel_bias_grad``)."""
    for n, t in (("q", q), ("k", k), ("v", v), ("out", out), ("dout", dout)):
        _check_bf16(n, t, 4)
    B, Nq, H, dqk = q.shape
    Nk = k.shape[1]
    _check_bwd(q, k, v, out, lse, dout, (B, H, Nq), (dq, dk, dv))
    scale = float(softmax_scale) if softmax_scale is not None else 1.0 / math.sqrt(dqk)
    dq, dk, dv = _grad_buffers(stream, (dq, q), (dk, k), (dv, v))
    p = AttnBwdParams()
    _fill_fwd(p.fwd, q, k, v, out, lse, _strides4, scale, causal)
    p.fwd.batch, p.fwd.seqlen_q, p.fwd.seqlen_k = B, Nq, Nk
    _fill_bwd(p, dout, dq, dk, dv, _strides4, deterministic, cta_pair, single_pass)
    _set_score_mod(p.fwd, q, softcap, alibi_slopes, rel_bias, rel_max_distance, rel_bidirectional)
    drel_bias = _rel_grad(drel_bias, rel_bias, rel_bias_grad, stream)
    p.drel_bias = _ptr(drel_bias)
    handles = _event_handles(phase_events)
    if handles is not None:
        for i, h in enumerate(handles):
            p.phase_events[i] = h
    ws, nbytes = _workspace(_lib.attn_bwd_workspace_size(ctypes.byref(p)), q.device, stream)
    _abi.check(_lib.attn_bwd(ctypes.byref(p), _ptr(ws), nbytes, _stream(stream, q.device)), "attn_bwd")
    return (dq, dk, dv) if rel_bias is None else (dq, dk, dv, drel_bias)


def attn_bwd_block_sparse(q, k, v, out, lse, dout, kv_count, kv_index, *, causal: bool = False,
                          softmax_scale: Optional[float] = None, deterministic: bool = False, dq=None, dk=None,
                          dv=None, softcap: Optional[float] = None, alibi_slopes: Optional[torch.Tensor] = None,
                          stream=None):
    """Block-sparse backward for :func:`attn_fwd_block_sparse` with the same kv_count / kv_index:
    returns (dQ, dK, dV) bf16 for the loss <O, dO>."""
    for n, t in (("q", q), ("k", k), ("v", v), ("out", out), ("dout", dout)):
        _check_bf16(n, t, 4)
    B, Nq, H, dqk = q.shape
    Nk = k.shape[1]
    _check_bwd(q, k, v, out, lse, dout, (B, H, Nq), (dq, dk, dv))
    max_kv, per_head = _check_lists(q, kv_count, kv_index)
    scale = float(softmax_scale) if softmax_scale is not None else 1.0 / math.sqrt(dqk)
    dq, dk, dv = _grad_buffers(stream, (dq, q), (dk, k), (dv, v))
    p = AttnBwdParams()
    _fill_fwd(p.fwd, q, k, v, out, lse, _strides4, scale, causal)
    p.fwd.batch, p.fwd.seqlen_q, p.fwd.seqlen_k = B, Nq, Nk
    _fill_bwd(p, dout, dq, dk, dv, _strides4, deterministic)
    _set_score_mod(p.fwd, q, softcap, alibi_slopes)
    ws, nbytes = _workspace(_lib.attn_bwd_block_sparse_workspace_size(ctypes.byref(p), per_head), q.device, stream)
    _abi.check(_lib.attn_bwd_block_sparse(ctypes.byref(p), _ptr(kv_count), _ptr(kv_index), max_kv, per_head,
                                          _ptr(ws), nbytes, _stream(stream, q.device)), "attn_bwd_block_sparse")
    return dq, dk, dv


def attn_bwd_varlen(q, k, v, out, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int, *,
                    causal: bool = False, softmax_scale: Optional[float] = None, deterministic: bool = False,
                    dq=None, dk=None, dv=None, stream=None, cta_pair: bool = False, softcap: Optional[float] = None,
                    alibi_slopes: Optional[torch.Tensor] = None, single_pass: bool = False,
                    rel_bias: Optional[torch.Tensor] = None, rel_max_distance: int = 128,
                    rel_bidirectional: bool = True, drel_bias: Optional[torch.Tensor] = None, rel_bias_grad: bool = True):
    """Packed variable-length backward: returns (dQ, dK, dV) packed like q, k, v; where query heads share
    K/V heads (attn_fwd_varlen), dK and dV are the sums over them. ``rel_bias`` and its gradient as in :func:`attn_bwd`."""
    ((tq, H, dqk), sq), (ks, sk), (vs, sv) = _bf16_layout("q", q, 3), _bf16_layout("k", k, 3), _bf16_layout("v", v, 3)
    (os, so), (ds, sd) = _bf16_layout("out", out, 3), _bf16_layout("dout", dout, 3)
    _check_offsets(q, cu_seqlens_q, cu_seqlens_k)
    dev = _check_packed_kv(q, k, v, H, dqk, ks, vs)
    want = (tq, H, vs[2])
    for n, t, shape in (("out", out, os), ("dout", dout, ds)):
        if shape != want or t.get_device() != dev:
            raise ValueError(f"{n} must be {want} on cuda:{dev}, got {tuple(shape)} on {t.device}")
    if lse.shape != (H, tq) or not lse.is_contiguous() or lse.dtype is not _F32 or lse.get_device() != dev:
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {(H, tq)} on cuda:{dev}")
    scale = float(softmax_scale) if softmax_scale is not None else 1.0 / math.sqrt(dqk)
    dq, tdq = _packed_grad("dq", dq, q, stream)
    dk, tdk = _packed_grad("dk", dk, k, stream)
    dv, tdv = _packed_grad("dv", dv, v, stream)
    drel_bias = _rel_grad(drel_bias, rel_bias, rel_bias_grad, stream)
    mod, rel = _mod_fields(q, softcap, alibi_slopes, rel_bias, rel_max_distance, rel_bidirectional)
    p = _pack_bwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
        0, sq[0], sq[1], 0, sk[0], sk[1], 0, sv[0], sv[1], 0, so[0], so[1],
        1, H, 0, 0, dqk, vs[2], cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), cu_seqlens_q.shape[0] - 1,
        int(max_seqlen_q), int(max_seqlen_k), tq, ks[0], scale, 1 if causal else 0, 0, 0, *mod,
        0, 0.0, 0.0, 0.0, 0, ks[1], *rel,
        dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
        0, sd[0], sd[1], 0, tdq[0], tdq[1], 0, tdk[0], tdk[1], 0, tdv[0], tdv[1],
        1 if deterministic else 0, 1 if cta_pair else 0, 0, 0, 0, 1 if single_pass else 0,
        drel_bias.data_ptr() if drel_bias is not None else 0)
    nbytes = _lib.attn_bwd_varlen_workspace_size(p)
    ws, ws_ptr = _workspace_ptr(nbytes, q, stream)
    status = _lib.attn_bwd_varlen(p, ws_ptr, nbytes, _stream_of(stream, q))
    if status:
        _abi.check(status, "attn_bwd_varlen")
    return (dq, dk, dv) if rel_bias is None else (dq, dk, dv, drel_bias)


def _check_table(t, device: int, num_seqs: int) -> int:
    """Row stride of a checked block table."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _I32 or not t.is_cuda or t.dim() != 2:
        raise ValueError("block_table must be an int32 CUDA tensor [requests, max_pages]")
    if t.get_device() != device:
        raise ValueError(f"block_table is on {t.device} but the call is on cuda:{device}")
    (rows, cols), (row, col) = t.shape, t.stride()
    if rows != num_seqs or cols < 1 or (col != 1 and cols > 1) or (rows > 1 and row < cols):
        raise ValueError(f"block_table must be [{num_seqs}, max_pages] with contiguous rows that do not overlap, got "
                         f"{tuple(t.shape)} with strides {t.stride()}")
    return max(row, cols)


def attn_kv_plan(seqlens_old: torch.Tensor, seqlens_new: torch.Tensor, block_table: torch.Tensor,
                 free_pages: torch.Tensor, free_count: torch.Tensor, page_size: int,
                 slot_mapping: Union[torch.Tensor, int], *, cu_seqlens_q: Optional[torch.Tensor] = None,
                 seqlens_k: Optional[torch.Tensor] = None, free_count_out: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None, stream=None):
    """Plans one step of a paged KV cache on the GPU (include/attn.h, attn_kv_plan): pages for every request's
    new tokens, and their slots. Request s holds ``seqlens_old[s]`` tokens and adds ``seqlens_new[s]`` (negative:
    it ends and returns its pages); its pages are listed in row s of ``block_table`` [requests, max_pages], and free
    ones on the stack ``free_pages[:free_count]``. The table, the stack and ``free_count`` (or ``free_count_out``,
    when given) are updated. ``slot_mapping`` is an int64 tensor, or the number of entries of one to make; entries
    past the step's tokens become -1. All other arrays are int32; ``positions``, when given, has as many entries as
    ``slot_mapping`` and gets each new token's position in its request (for :func:`attn_kv_append_rotary`), then -1.
    Returns (cu_seqlens_q [requests + 1], seqlens_k [requests], slot_mapping, status [1]): status 0, or 1 (too few
    free pages), 2 (a row of the table is too short), 3 (slot_mapping is), 4 (free_pages is), and then nothing is
    changed and the step holds no tokens."""
    if not isinstance(seqlens_old, torch.Tensor) or not seqlens_old.is_cuda:
        raise ValueError("seqlens_old must be a contiguous int32 CUDA tensor")
    n, dev = seqlens_old.numel(), seqlens_old.get_device()
    if n < 1:
        raise ValueError("attn_kv_plan needs at least one request")
    _check_int32("seqlens_old", seqlens_old, dev, n)
    _check_int32("seqlens_new", seqlens_new, dev, n)
    _check_int32("free_pages", free_pages, dev, -1)
    _check_int32("free_count", free_count, dev, 1)
    table_stride = _check_table(block_table, dev, n)

    def given(name, t, size):
        if t is None:
            t = torch.empty((size,), dtype=_I32, device=seqlens_old.device)
            _used_on(stream, t)
        else:
            _check_int32(name, t, dev, size)
        return t

    cu_seqlens_q, seqlens_k = given("cu_seqlens_q", cu_seqlens_q, n + 1), given("seqlens_k", seqlens_k, n)
    status = given("status", status, 1)
    free_count_out = free_count if free_count_out is None else given("free_count_out", free_count_out, 1)
    if isinstance(slot_mapping, int):
        slot_mapping = torch.empty((slot_mapping,), dtype=_I64, device=seqlens_old.device)
        _used_on(stream, slot_mapping)
    elif slot_mapping.dtype is not _I64 or slot_mapping.dim() != 1 or not slot_mapping.is_contiguous() or \
            not slot_mapping.is_cuda or slot_mapping.get_device() != dev:
        raise ValueError(f"slot_mapping must be a contiguous int64 tensor [max_tokens] on cuda:{dev}")
    if positions is not None:
        _check_int32("positions", positions, dev, slot_mapping.shape[0])
    p = _pack_plan(seqlens_old.data_ptr(), seqlens_new.data_ptr(), block_table.data_ptr(), table_stride,
                   free_pages.data_ptr(), free_count.data_ptr(), free_count_out.data_ptr(), cu_seqlens_q.data_ptr(),
                   seqlens_k.data_ptr(), slot_mapping.data_ptr(), status.data_ptr(),
                   n, block_table.shape[1], int(page_size), free_pages.shape[0], slot_mapping.shape[0],
                   0 if positions is None else positions.data_ptr())
    st = _lib.attn_kv_plan(p, _stream_of(stream, seqlens_old))
    if st:
        _abi.check(st, "attn_kv_plan")
    return cu_seqlens_q, seqlens_k, slot_mapping, status


def _cache_layout(k_cache, v_cache, device: int):
    """Layouts of checked caches [pages, page_size, Hkv, d]."""
    (ks, kt), (vs, vt) = _bf16_layout("k_cache", k_cache, 4), _bf16_layout("v_cache", v_cache, 4)
    if ks[:3] != vs[:3]:
        raise ValueError(f"k_cache {tuple(ks)} and v_cache {tuple(vs)} must be [pages, page_size, Hkv, d] alike but for d")
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.get_device() != device:
            raise ValueError(f"{n} is on {t.device} but the call is on cuda:{device}")
    return ks, kt, vs, vt


def attn_kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   slot_mapping: torch.Tensor, *, stream=None) -> None:
    """Writes new tokens' k [tokens, Hkv, d_qk] and v [tokens, Hkv, d_v] into the paged caches k_cache [pages,
    page_size, Hkv, d_qk] and v_cache [pages, page_size, Hkv, d_v] (bf16, any strides with contiguous d): row i goes
    to slot ``slot_mapping[i]`` (int64; page slot // page_size, row slot % page_size). Slots outside the cache, as -1,
    write nothing; slots must differ."""
    p, _ = _append_fields(k, v, k_cache, v_cache, slot_mapping)
    st = _lib.attn_kv_append(_pack_append(*p), _stream_of(stream, k))
    if st:
        _abi.check(st, "attn_kv_append")


def _append_fields(k, v, k_cache, v_cache, slot_mapping):
    """The fields of a checked append (attn_kv_append_params), and k's shape."""
    (ks, kt), (vs, vt) = _bf16_layout("k", k, 3), _bf16_layout("v", v, 3)
    dev = k.get_device()
    kcs, kct, vcs, vct = _cache_layout(k_cache, v_cache, dev)
    if vs[:2] != ks[:2] or v.get_device() != dev:
        raise ValueError(f"shape or device mismatch k{tuple(ks)} v{tuple(vs)}")
    if kcs[2:] != ks[1:] or vcs[2:] != vs[1:]:
        raise ValueError(f"k_cache {tuple(kcs)} and v_cache {tuple(vcs)} do not hold rows of k {tuple(ks)} and v {tuple(vs)}")
    if slot_mapping.dtype is not _I64 or slot_mapping.dim() != 1 or slot_mapping.shape[0] != ks[0] or \
            not slot_mapping.is_contiguous() or not slot_mapping.is_cuda or slot_mapping.get_device() != dev:
        raise ValueError(f"slot_mapping must be a contiguous int64 tensor [{ks[0]}] on cuda:{dev}")
    return (k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), kt[0], kt[1], vt[0], vt[1],
            kct[0], kct[1], kct[2], vct[0], vct[1], vct[2], slot_mapping.data_ptr(),
            ks[0], ks[1], ks[2], vs[2], kcs[1], kcs[0]), ks


def _no_table_gradient(cos, sin):
    for name, t in (("cos", cos), ("sin", sin)):
        if isinstance(t, torch.Tensor) and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} has no gradient here: pass it detached")


def _check_rotation(cos, sin, device: int, rotary_offset: int, head: int):
    """The checked tables' fields: pointers, row stride, positions, rotary_dim."""
    for name, t in (("cos", cos), ("sin", sin)):
        if not isinstance(t, torch.Tensor) or t.dtype is not _F32 or not t.is_cuda or t.dim() != 2:
            raise ValueError(f"{name} must be a float32 CUDA tensor [positions, rotary_dim / 2] with contiguous rows")
        if t.get_device() != device:
            raise ValueError(f"{name} is on {t.device} but the call is on cuda:{device}")
    (n, half), (row, col) = cos.shape, cos.stride()
    if sin.shape != cos.shape or (n > 1 and sin.stride() != (row, col)) or col != 1 or sin.stride(1) != 1:
        raise ValueError(f"cos {tuple(cos.shape)} and sin {tuple(sin.shape)} must be alike, strides too, with contiguous rows")
    if half < 8 or half % 8 or rotary_offset < 0 or rotary_offset % 8:
        raise ValueError(f"rotary_dim {2 * half} must be a multiple of 16 and rotary_offset {rotary_offset} of 8")
    if rotary_offset + 2 * half > head:
        raise ValueError(f"columns {rotary_offset} .. {rotary_offset + 2 * half - 1} are not all of a head of {head}")
    return cos.data_ptr(), sin.data_ptr(), row if n > 1 else half, n, 2 * half


def attn_kv_append_rotary(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                          v_cache: torch.Tensor, slot_mapping: torch.Tensor, positions: torch.Tensor, cos: torch.Tensor,
                          sin: torch.Tensor, *, rotary_offset: int = 0, interleaved: bool = False,
                          q_out: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """:func:`attn_kv_append` with the rotation of :func:`attn_rotary` on the way: k's row i, rotated by
    ``positions[i]`` (int32 [tokens], as :func:`attn_kv_plan` writes it), and v's go to slot ``slot_mapping[i]``, and q
    [tokens, H, d_qk], unless None, is rotated into ``q_out`` (which may be q; made when not given). A token whose
    position lies outside the tables writes nothing, one whose slot is outside the cache only its row of q_out.
    Returns q_out (None without q)."""
    _no_table_gradient(cos, sin)
    append, ks = _append_fields(k, v, k_cache, v_cache, slot_mapping)
    dev = k.get_device()
    _check_int32("positions", positions, dev, ks[0])
    cos_ptr, sin_ptr, row, n, dim = _check_rotation(cos, sin, dev, rotary_offset, ks[2])
    heads, qt, qo, q_ptr, out_ptr = 0, (0, 0), (0, 0), 0, 0
    if q is not None:
        qs, qt = _bf16_layout("q", q, 3)
        if qs[0] != ks[0] or qs[2] != ks[2] or q.get_device() != dev:
            raise ValueError(f"q {tuple(qs)} does not match k {tuple(ks)} on cuda:{dev}")
        q_out, qo = _rotated("q_out", q_out, q, qs, stream)
        heads, q_ptr, out_ptr = qs[1], q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    p = _pack_append_rotary(*append, q_ptr, out_ptr, qt[0], qt[1], qo[0], qo[1], positions.data_ptr(), cos_ptr, sin_ptr, row,
                            heads, dim, rotary_offset, 1 if interleaved else 0, n)
    st = _lib.attn_kv_append_rotary(p, _stream_of(stream, k))
    if st:
        _abi.check(st, "attn_kv_append_rotary")
    return q_out


def _rotated(name: str, out, like, shape, stream):
    """An output buffer for the rotated `like` (the given one, checked) and its strides, the last one left out."""
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=like.device)
        if stream is not None:
            _used_on(stream, out)
        row = shape[-2] * shape[-1]
        return out, (row, shape[-1]) if len(shape) == 3 else (shape[1] * row, row, shape[-1])
    if out.shape != shape or out.get_device() != like.get_device():
        raise ValueError(f"{name} must be {tuple(shape)} on {like.device}, got {tuple(out.shape)} on {out.device}")
    return out, _bf16_layout(name, out, len(shape))[1][:-1]


def attn_rotary(q: torch.Tensor, k: Optional[torch.Tensor], cos: torch.Tensor, sin: torch.Tensor,
                positions: Optional[torch.Tensor] = None, *, rotary_offset: int = 0, interleaved: bool = False,
                inverse: bool = False, q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Rotary position encoding of q [B, N, H, d_qk] and, unless None, k [B, N, Hkv, d_qk] (or packed, [total, H, d_qk];
    bf16): pairs of columns of ``rotary_offset .. rotary_offset + rotary_dim - 1`` of every head turn by their row's
    position p, (x, y) -> (x c - y s, x s + y c) with c = cos[p, f] and s = sin[p, f] (float32 [positions,
    rotary_dim / 2]); pair f is columns f and f + rotary_dim / 2, or with ``interleaved`` 2f and 2f + 1. ``positions``
    is int32 [B, N] or [N] ([total]); without it a row's position is its index. ``inverse`` turns back: of the
    gradients of the outputs it gives those of the inputs. q_out and k_out may be q and k. Rows whose position lies
    outside the tables are not written. Returns (q_out, k_out)."""
    _no_table_gradient(cos, sin)
    dim = 3 if isinstance(q, torch.Tensor) and q.dim() == 3 else 4
    qs, qt = _bf16_layout("q", q, dim)
    dev = q.get_device()
    cos_ptr, sin_ptr, row, n_pos, rot = _check_rotation(cos, sin, dev, rotary_offset, qs[-1])
    heads_kv = k_ptr = ko_ptr = 0
    if k is not None:
        ks, kt = _bf16_layout("k", k, dim)
        if ks[:-2] != qs[:-2] or ks[-1] != qs[-1] or k.get_device() != dev:
            raise ValueError(f"k {tuple(ks)} does not match q {tuple(qs)} on cuda:{dev}")
        k_out, ko = _rotated("k_out", k_out, k, ks, stream)
        heads_kv, k_ptr, ko_ptr = ks[-2], k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    else:
        kt = ko = (0, 0, 0)
    q_out, qo = _rotated("q_out", q_out, q, qs, stream)
    if dim == 4:
        batch, n = qs[0], qs[1]
        strides = (*qt[:3], *kt[:3], *qo, *ko)
    else:
        batch, n = 1, qs[0]
        strides = (0, qt[0], qt[1], 0, kt[0], kt[1], 0, qo[0], qo[1], 0, ko[0], ko[1])
    pos_ptr = pos_batch = 0
    if positions is not None:
        if dim == 4 and positions.dim() == 2:
            if positions.shape != (batch, n):
                raise ValueError(f"positions must be [{batch}, {n}] or [{n}], got {tuple(positions.shape)}")
            _check_int32("positions", positions.view(-1) if positions.is_contiguous() else positions, dev, batch * n)
            pos_batch = n
        else:
            _check_int32("positions", positions, dev, n)
        pos_ptr = positions.data_ptr()
    elif n > n_pos:
        raise ValueError(f"{n} rows but the tables hold {n_pos} positions")
    p = _pack_rotary(q.data_ptr(), k_ptr, q_out.data_ptr(), ko_ptr, *strides, pos_ptr, pos_batch, cos_ptr, sin_ptr, row, batch,
                     n, qs[-2], heads_kv, qs[-1], rot, rotary_offset, 1 if interleaved else 0, 1 if inverse else 0, n_pos)
    st = _lib.attn_rotary(p, _stream_of(stream, q))
    if st:
        _abi.check(st, "attn_rotary")
    return q_out, k_out


def attn_fwd_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                   cu_seqlens_q: torch.Tensor, seqlens_k: torch.Tensor, max_seqlen_q: int, *, causal: bool = True,
                   softmax_scale: Optional[float] = None, softcap: Optional[float] = None,
                   alibi_slopes: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, rel_bias: Optional[torch.Tensor] = None, rel_max_distance: int = 128,
                   rel_bidirectional: bool = True, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of new tokens over a paged KV cache (include/attn.h, attn_fwd_paged). q [total_q, H, d_qk] (bf16)
    packs the requests' new tokens, request s's in rows cu_seqlens_q[s] .. cu_seqlens_q[s + 1] - 1 (one for a decoding
    request, a chunk for a prompt, or none); its keys are the first seqlens_k[s] tokens on the pages of row s of
    ``block_table`` [requests, max_pages], the new ones among them, in k_cache [pages, page_size, Hkv, d_qk] and
    v_cache [pages, page_size, Hkv, d_v]; Hkv divides H. With ``causal`` (the default) query i of n sees the keys up
    to position i + seqlens_k[s] - n. cu_seqlens_q [requests + 1], seqlens_k [requests] and the table are int32 on
    q's GPU; ``max_seqlen_q`` bounds the queries of a request (of one with more the first are computed). Score
    modifications as in :func:`attn_fwd`.
    Returns (O [total_q, H, d_v] bf16, LSE [H, total_q] fp32); rows behind the last request are not written."""
    (tq, H, dqk), sq = _bf16_layout("q", q, 3)
    dev = q.get_device()
    ks, kt, vs, vt = _cache_layout(k_cache, v_cache, dev)
    hk, dv = ks[2], vs[3]
    if ks[3] != dqk:
        raise ValueError(f"k_cache {tuple(ks)} does not match q {tuple(q.shape)}")
    if hk < 1 or H % hk != 0:
        raise ValueError(f"{hk} K/V heads do not divide {H} query heads")
    _check_int32("seqlens_k", seqlens_k, dev, -1)
    n = seqlens_k.shape[0]
    _check_int32("cu_seqlens_q", cu_seqlens_q, dev, n + 1)
    table_stride = _check_table(block_table, dev, n)
    if out is None:
        out = torch.empty((tq, H, dv), dtype=_BF16, device=q.device)
        so = (H * dv, dv)
    else:
        shape, so = _bf16_layout("out", out, 3)
        if shape != (tq, H, dv) or out.get_device() != dev:
            raise ValueError(f"out must be {(tq, H, dv)} on cuda:{dev}, got {tuple(shape)} on {out.device}")
    if lse is None:
        lse = torch.empty((H, tq), dtype=_F32, device=q.device)
    elif lse.shape != (H, tq) or not lse.is_contiguous() or lse.dtype is not _F32 or lse.device != q.device:
        raise ValueError(f"lse must be a contiguous float32 [H, total_q] tensor on cuda:{dev}")
    mod, rel = _mod_fields(q, softcap, alibi_slopes, rel_bias, rel_max_distance, rel_bidirectional)
    p = _pack_paged(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), lse.data_ptr(),
                    sq[0], sq[1], so[0], so[1], kt[0], kt[1], kt[2], vt[0], vt[1], vt[2],
                    block_table.data_ptr(), table_stride, cu_seqlens_q.data_ptr(), seqlens_k.data_ptr(),
                    n, H, hk, dqk, dv, ks[1], ks[0], block_table.shape[1], tq, int(max_seqlen_q),
                    float(softmax_scale) if softmax_scale is not None else 1.0 / math.sqrt(dqk),
                    1 if causal else 0, *mod, *rel)
    nbytes = _lib.attn_fwd_paged_workspace_size(p)
    ws, ws_ptr = _workspace_ptr(nbytes, q, stream)
    if stream is not None:
        _used_on(stream, out, lse)
    st = _lib.attn_fwd_paged(p, ws_ptr, nbytes, _stream_of(stream, q))
    if st:
        _abi.check(st, "attn_fwd_paged")
    return out, lse


def attn_exp2_eval(x: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Evaluates the kernels' software (Cody-Waite + cubic) and hardware exp2 on a float32 CUDA tensor."""
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 CUDA tensor")
    yp, yh = torch.empty_like(x), torch.empty_like(x)
    _abi.check(_lib.attn_exp2_eval(_ptr(x), _ptr(yp), _ptr(yh), x.numel(), _stream(stream)), "attn_exp2_eval")
    return yp, yh


def attn_get_device_status(stream=None) -> int:
    """Synchronises the stream; raises AttnError(ATTN_ERR_TIMEOUT) if a kernel recorded a failure."""
    detail = ctypes.c_uint32(0)
    st = _lib.attn_get_device_status(_stream(stream), ctypes.byref(detail))
    if st != _abi.ATTN_OK:
        raise AttnError(st, f"device status 0x{detail.value:08x}")
    return detail.value


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, rel_bias, causal, softmax_scale, deterministic, kv_count, kv_index, mod, rel):
        if kv_count is None:
            o, lse = attn_fwd(q, k, v, causal=causal, softmax_scale=softmax_scale, rel_bias=rel_bias, **mod, **rel)
        else:
            if rel_bias is not None:
                raise ValueError("block_mask and rel_bias do not go together")
            o, lse = attn_fwd_block_sparse(q, k, v, kv_count, kv_index, causal=causal, softmax_scale=softmax_scale,
                                           **mod)
        ctx.save_for_backward(q, k, v, o, lse, rel_bias)
        ctx.causal, ctx.scale, ctx.det = causal, softmax_scale, deterministic
        ctx.lists = (kv_count, kv_index)
        ctx.mod, ctx.rel = mod, rel
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse, rel_bias = ctx.saved_tensors
        kv_count, kv_index = ctx.lists
        if kv_count is None:
            grads = attn_bwd(q, k, v, o, lse, do.contiguous(), causal=ctx.causal, softmax_scale=ctx.scale,
                             deterministic=ctx.det, rel_bias=rel_bias, rel_bias_grad=ctx.needs_input_grad[3], **ctx.mod,
                             **ctx.rel)
        else:
            grads = attn_bwd_block_sparse(q, k, v, o, lse, do.contiguous(), kv_count, kv_index,
                                          causal=ctx.causal, softmax_scale=ctx.scale, deterministic=ctx.det,
                                          **ctx.mod)
        return (*grads, *(None,) * (11 - len(grads)))


def attention(q, k, v, causal: bool = False, softmax_scale: Optional[float] = None, deterministic: bool = False,
              block_mask: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, softcap: Optional[float] = None,
              alibi_slopes: Optional[torch.Tensor] = None, rel_bias: Optional[torch.Tensor] = None, rel_max_distance: int = 128,
              rel_bidirectional: bool = True):
    """Autograd wrapper over attn_fwd / attn_bwd for [B, N, H, d] bf16 tensors; k and v may have fewer
    heads, a divisor of H, shared among the query heads as in attn_fwd. ``block_mask``
    = (kv_count, kv_index) selects the block-sparse pair attn_fwd_block_sparse / attn_bwd_block_sparse;
    ``softcap`` / ``alibi_slopes`` / ``rel_bias`` (which gets a gradient; not with block_mask) a score modification."""
    kv_count, kv_index = block_mask if block_mask is not None else (None, None)
    return _Attention.apply(q, k, v, rel_bias, causal, softmax_scale, deterministic, kv_count, kv_index,
                            dict(softcap=softcap, alibi_slopes=alibi_slopes),
                            dict(rel_max_distance=rel_max_distance, rel_bidirectional=rel_bidirectional))


class _AttentionVarlen(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, rel_bias, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal, softmax_scale,
                deterministic, mod):
        o, lse = attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal=causal,
                                 softmax_scale=softmax_scale, rel_bias=rel_bias, **mod)
        ctx.save_for_backward(q, k, v, o, lse, rel_bias, cu_seqlens_q, cu_seqlens_k)
        ctx.lengths = (max_seqlen_q, max_seqlen_k)
        ctx.causal, ctx.scale, ctx.det, ctx.mod = causal, softmax_scale, deterministic, mod
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse, rel_bias, cu_q, cu_k = ctx.saved_tensors
        grads = attn_bwd_varlen(q, k, v, o, lse, do.contiguous(), cu_q, cu_k, *ctx.lengths, causal=ctx.causal,
                                softmax_scale=ctx.scale, deterministic=ctx.det, rel_bias=rel_bias,
                                rel_bias_grad=ctx.needs_input_grad[3], **ctx.mod)
        return (*grads, *(None,) * (12 - len(grads)))


def attention_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int, causal: bool = False,
                     softmax_scale: Optional[float] = None, deterministic: bool = False,
                     softcap: Optional[float] = None, alibi_slopes: Optional[torch.Tensor] = None,
                     rel_bias: Optional[torch.Tensor] = None, rel_max_distance: int = 128,
                     rel_bidirectional: bool = True):
    """Autograd wrapper over attn_fwd_varlen / attn_bwd_varlen for packed bf16 tensors q [total_q, H, d_qk],
    k [total_k, Hkv, d_qk] and v [total_k, Hkv, d_v]; ``softcap`` / ``alibi_slopes`` / ``rel_bias`` (which gets a gradient)
    select a score modification.
    The offsets cover every row: cu_seqlens[-1] is the total (of a buffer with spare rows, pass the used part: O and the
    gradients of rows behind the last offset are not written)."""
    return _AttentionVarlen.apply(q, k, v, rel_bias, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal,
                                  softmax_scale, deterministic,
                                  dict(softcap=softcap, alibi_slopes=alibi_slopes, rel_max_distance=rel_max_distance,
                                       rel_bidirectional=rel_bidirectional))


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, cos, sin, positions, rotary_offset, interleaved):
        ctx.save_for_backward(cos, sin, positions)
        ctx.how = dict(rotary_offset=rotary_offset, interleaved=interleaved)
        out = attn_rotary(q, k, cos, sin, positions, **ctx.how)
        return out if k is not None else out[0]

    @staticmethod
    def backward(ctx, dq, dk=None):
        cos, sin, positions = ctx.saved_tensors
        dq, dk = attn_rotary(dq.contiguous(), dk.contiguous() if dk is not None else None, cos, sin, positions, inverse=True,
                             **ctx.how)
        return dq, dk, None, None, None, None, None


def rotary(q, k, cos, sin, positions: Optional[torch.Tensor] = None, rotary_offset: int = 0, interleaved: bool = False):
    """Autograd wrapper over attn_rotary: (q, k) rotated, or q alone where k is None. Every row needs a position inside
    the tables (rows without one are not written). The tables get no gradient; ones that ask for it are refused."""
    _no_table_gradient(cos, sin)  # (inside the function no gradients are recorded)
    return _Rotary.apply(q, k, cos, sin, positions, rotary_offset, interleaved)
