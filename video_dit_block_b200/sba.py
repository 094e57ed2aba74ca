"""Python binding of the C ABI in include/sba.h (argument marshalling only).

Every function takes torch CUDA tensors, allocates outputs with torch (device
memory and streams are PyTorch's job here), and calls the CUDA library through
ctypes.  There is no fallback: if libsba.so is missing or a tensor is not on a
CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

from .build import LIB

SBA_OK = 0
_STATUS = {0: "SBA_OK", 1: "SBA_ERR_INVALID_ARG", 2: "SBA_ERR_UNSUPPORTED", 3: "SBA_ERR_ALIGNMENT",
           4: "SBA_ERR_CUDA", 5: "SBA_ERR_TIMEOUT", 6: "SBA_ERR_DEVICE_FLAG",
           7: "SBA_ERR_SCRATCH_TOO_SMALL"}
MAX_NPAD = 262144
BLOCK = 64


class SbaError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {_STATUS.get(code, code)} ({_lib.sba_strerror(code).decode()})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libsba.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError(f"CUDA library not built: {LIB} is missing "
                               "(run `python -m video_dit_block_b200.build`)")
        L = ctypes.CDLL(LIB)
        vp, i32, f64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_double, ctypes.c_float, ctypes.c_size_t
        L.sba_keep_count.restype = ctypes.c_int32
        L.sba_keep_count.argtypes = [ctypes.c_int32, f64]
        L.sba_pool_select_workspace_size.restype = sz
        L.sba_pool_select_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.sba_pool_select.restype = i32
        L.sba_pool_select.argtypes = [vp, vp, i32, i32, i32, i32, vp, i32, f64, i32, vp, vp, vp, sz, vp]
        L.sba_pool_select_lse_workspace_size.restype = sz
        L.sba_pool_select_lse_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.sba_pool_select_lse.restype = i32
        L.sba_pool_select_lse.argtypes = [vp, vp, i32, i32, i32, i32, vp, i32, i32, f64, i32, i32, vp, vp, vp,
                                          sz, vp]
        L.sba_qk_norm_rope_pool.restype = i32
        L.sba_qk_norm_rope_pool.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, i32, i32, f64, f32, vp, vp, vp]
        L.sba_pool_select_means.restype = i32
        L.sba_pool_select_means.argtypes = [vp, vp, i32, i32, i32, i32, vp, i32, f64, i32, vp, vp, vp, sz, vp]
        L.sba_keep_count_budget.restype = ctypes.c_int32
        L.sba_keep_count_budget.argtypes = [ctypes.c_int32, f64, ctypes.c_int32]
        L.sba_mean_compensation_workspace_size.restype = sz
        L.sba_mean_compensation_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.sba_attention_mean_compensated.restype = i32
        L.sba_attention_mean_compensated.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, i32, vp, vp, i32,
                                                     vp, f32, vp, sz, vp]
        L.sba_attention_compensated.restype = i32
        L.sba_attention_compensated.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, i32, vp, vp, i32, vp,
                                                f32, vp]
        L.sba_block_means.restype = i32
        L.sba_block_means.argtypes = [vp, i32, i32, i32, i32, vp, i32, vp, vp]
        L.sba_attention.restype = i32
        L.sba_attention.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, i32, vp, vp, i32, f32, vp]
        L.sba_pair_workspace_size.restype = sz
        L.sba_pair_workspace_size.argtypes = [i32, i32, i32, i32]
        L.sba_pair_query_blocks.restype = i32
        L.sba_pair_query_blocks.argtypes = [vp, vp, i32, i32, i32, i32, vp, i32, vp, vp, sz, vp]
        L.sba_attention_paired.restype = i32
        L.sba_attention_paired.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, i32, vp, vp, i32, vp,
                                           f32, vp]
        L.sba_dense_attention.restype = i32
        L.sba_dense_attention.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, f32, vp]
        L.sba_attention_to_shards.restype = i32
        L.sba_attention_to_shards.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, i32,
                                              vp, vp, i32, vp, f32, vp]
        L.sba_get_device_status.restype = i32
        L.sba_get_device_status.argtypes = [vp]
        L.sba_set_wait_limit.restype = None
        L.sba_set_wait_limit.argtypes = [ctypes.c_uint64]
        L.sba_set_attention_kernel.restype = i32
        L.sba_set_attention_kernel.argtypes = [i32]
        L.sba_pool_select_noalloc.restype = i32
        L.sba_pool_select_noalloc.argtypes = [vp, vp, i32, i32, i32, i32, vp, i32, f64, i32, vp, vp, vp]
        L.sba_noalloc_scratch_bytes.restype = sz
        L.sba_noalloc_scratch_bytes.argtypes = []
        L.sba_keep_token_count.restype = ctypes.c_int32
        L.sba_keep_token_count.argtypes = [ctypes.c_int32, f64]
        L.sba_token_prune_workspace_size.restype = sz
        L.sba_token_prune_workspace_size.argtypes = [i32, i32]
        L.sba_token_prune_select.restype = i32
        L.sba_token_prune_select.argtypes = [vp, i32, i32, i32, vp, f64, i32, vp, vp, vp, sz, vp]
        L.sba_gather_tokens.restype = i32
        L.sba_gather_tokens.argtypes = [vp, i32, i32, i32, i32, vp, vp, i32, vp, vp]
        L.sba_residual_norm.restype = i32
        L.sba_residual_norm.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, i32, vp, vp, i32, vp, vp, vp,
                                        vp, i32, i32, vp, f32, vp]
        L.sba_token_quantize.restype = i32
        L.sba_token_quantize.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp]
        L.sba_int8_linear.restype = i32
        L.sba_int8_linear.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, i32, i32, vp, i32, vp, vp, i32, i32, vp,
                                      vp]
        L.sba_int8_linear_plan.restype = i32
        L.sba_int8_linear_plan.argtypes = [ctypes.c_longlong, i32, i32, i32, ctypes.POINTER(i32), ctypes.POINTER(i32)]
        L.sba_rotary.restype = i32
        L.sba_rotary.argtypes = [vp, vp, i32, vp, i32, i32, i32, i32, i32, vp, i32, i32, vp, vp, f32, i32, vp]
        L.sba_strerror.restype = ctypes.c_char_p
        L.sba_strerror.argtypes = [i32]
        _lib = L
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _raw(t):
    """The address of an optional tensor, as the plain integer that ctypes takes for a void *."""
    return None if t is None else t.data_ptr()


def _check(code, what):
    if code != SBA_OK:
        raise SbaError(code, what)


def _qkv(*ts):
    for t in ts:
        if not (t.is_cuda and t.dtype == torch.bfloat16 and t.dim() == 4 and t.is_contiguous()):
            raise ValueError("expected contiguous bf16 CUDA tensors [B, H, Npad, D]")
    return ts[0].shape


def _valid_len(valid_len, device):
    if valid_len is None:
        return None
    if not (valid_len.is_cuda and valid_len.dtype == torch.int32 and valid_len.is_contiguous()):
        raise ValueError("valid_len must be a contiguous int32 CUDA tensor [B]")
    return valid_len


def keep_count(n_blocks: int, sparsity: float) -> int:
    return int(lib().sba_keep_count(int(n_blocks), float(sparsity)))


def kmax_for(Npad: int, sparsity: float, block: int = BLOCK) -> int:
    """Row capacity of kv_idx that every sample of padded length Npad fits in."""
    return keep_count(Npad // block, sparsity)


def workspace_size(B: int, H: int, Npad: int, D: int, block: int = BLOCK) -> int:
    return int(lib().sba_pool_select_workspace_size(B, H, Npad, D, block))


def pool_select(q, k, valid_len=None, sparsity: float = 0.0, kmax: int | None = None,
                block: int = BLOCK, kv_idx=None, kv_cnt=None, workspace=None, stream=None):
    """Routing: returns (kv_idx int32 [B,H,Npad/64,kmax], kv_cnt int32 [B,H,Npad/64])."""
    B, H, Npad, D = _qkv(q, k)
    vl = _valid_len(valid_len, q.device)
    nB = Npad // block
    if kmax is None:
        kmax = kmax_for(Npad, sparsity, block)
    if kv_idx is None:
        kv_idx = torch.empty((B, H, nB, kmax), dtype=torch.int32, device=q.device)
    if kv_cnt is None:
        kv_cnt = torch.empty((B, H, nB), dtype=torch.int32, device=q.device)
    wsz = workspace_size(B, H, Npad, D, block)
    if workspace is None:
        workspace = torch.empty(wsz, dtype=torch.uint8, device=q.device)
    _check(lib().sba_pool_select(_ptr(q), _ptr(k), B, H, Npad, D, _ptr(vl), block, float(sparsity),
                                 int(kmax), _ptr(kv_idx), _ptr(kv_cnt), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)),
           "sba_pool_select")
    return kv_idx, kv_cnt


def keep_count_budget(n_blocks: int, sparsity: float, budget: int = 1) -> int:
    """keep(n, s) rounded up to a multiple of `budget`, at most n (sba_keep_count_budget)."""
    if budget < 1:
        raise ValueError("budget must be >= 1")
    return int(lib().sba_keep_count_budget(int(n_blocks), float(sparsity), int(budget)))


def lse_workspace_size(B: int, H: int, Npad: int, D: int, nsub: int = 4, block: int = BLOCK) -> int:
    return int(lib().sba_pool_select_lse_workspace_size(B, H, Npad, D, block, nsub))


def pool_select_lse(q, k, valid_len=None, sparsity: float = 0.0, nsub: int = 4, budget: int = 1,
                    kmax: int | None = None, block: int = BLOCK, kv_idx=None, kv_cnt=None, workspace=None,
                    stream=None):
    """Sub-block log-sum-exp routing: (kv_idx int32 [B,H,Npad/64,kmax], kv_cnt int32 [B,H,Npad/64])."""
    B, H, Npad, D = _qkv(q, k)
    vl = _valid_len(valid_len, q.device)
    nB = Npad // block
    if kmax is None:
        kmax = keep_count_budget(nB, sparsity, budget)
    if kv_idx is None:
        kv_idx = torch.empty((B, H, nB, kmax), dtype=torch.int32, device=q.device)
    if kv_cnt is None:
        kv_cnt = torch.empty((B, H, nB), dtype=torch.int32, device=q.device)
    if workspace is None:
        workspace = torch.empty(lse_workspace_size(B, H, Npad, D, nsub, block), dtype=torch.uint8,
                                device=q.device)
    _check(lib().sba_pool_select_lse(_ptr(q), _ptr(k), B, H, Npad, D, _ptr(vl), block, int(nsub),
                                     float(sparsity), int(budget), int(kmax), _ptr(kv_idx), _ptr(kv_cnt),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream(stream)), "sba_pool_select_lse")
    return kv_idx, kv_cnt


def qk_norm_rope_pool(x, weight, pos, valid_len=None, rope_dim: int = 96, rope_base: float = 10000.0,
                      eps: float = 1e-6, out=None, means=None, want_means: bool = True, block: int = BLOCK,
                      stream=None):
    """QK RMSNorm + 3D RoPE (see include/sba.h), with the block means of the output.
    weight: bf16 [D]; pos: int32 [B, Npad, 3].  Returns (out bf16, means fp64 or None)."""
    B, H, Npad, D = _qkv(x)
    if not (weight.is_cuda and weight.dtype == torch.bfloat16 and weight.shape == (D,) and weight.is_contiguous()):
        raise ValueError("weight must be a contiguous bf16 CUDA tensor [D]")
    if not (pos.is_cuda and pos.dtype == torch.int32 and pos.shape == (B, Npad, 3) and pos.is_contiguous()):
        raise ValueError("pos must be a contiguous int32 CUDA tensor [B, Npad, 3]")
    if out is None:
        out = torch.empty_like(x)
    if means is None and want_means:
        means = torch.empty((B, H, Npad // block, D), dtype=torch.float64, device=x.device)
    _check(lib().sba_qk_norm_rope_pool(_ptr(x), _ptr(weight), _ptr(pos), B, H, Npad, D,
                                       _ptr(_valid_len(valid_len, x.device)), block, int(rope_dim),
                                       float(rope_base), float(eps), _ptr(out), _ptr(means), _stream(stream)),
           "sba_qk_norm_rope_pool")
    return out, means


def pool_select_means(qmean, kmean, valid_len=None, sparsity: float = 0.0, kmax: int | None = None,
                      block: int = BLOCK, kv_idx=None, kv_cnt=None, workspace=None, stream=None):
    """Routing from given fp64 block means [B, H, Npad/64, D] (no pass over Q and K)."""
    B, H, nB, D = qmean.shape
    for t in (qmean, kmean):
        if not (t.is_cuda and t.dtype == torch.float64 and t.is_contiguous() and t.shape == (B, H, nB, D)):
            raise ValueError("qmean / kmean must be contiguous fp64 CUDA tensors [B, H, Npad/64, D]")
    Npad = nB * block
    vl = _valid_len(valid_len, qmean.device)
    if kmax is None:
        kmax = kmax_for(Npad, sparsity, block)
    if kv_idx is None:
        kv_idx = torch.empty((B, H, nB, kmax), dtype=torch.int32, device=qmean.device)
    if kv_cnt is None:
        kv_cnt = torch.empty((B, H, nB), dtype=torch.int32, device=qmean.device)
    if workspace is None:
        workspace = torch.empty(workspace_size(B, H, Npad, D, block), dtype=torch.uint8, device=qmean.device)
    _check(lib().sba_pool_select_means(_ptr(qmean), _ptr(kmean), B, H, Npad, D, _ptr(vl), block, float(sparsity),
                                       int(kmax), _ptr(kv_idx), _ptr(kv_cnt), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream)),
           "sba_pool_select_means")
    return kv_idx, kv_cnt


def block_means(x, valid_len=None, block: int = BLOCK, stream=None):
    """fp64 block means [B, H, Npad/64, D]."""
    B, H, Npad, D = _qkv(x)
    out = torch.empty((B, H, Npad // block, D), dtype=torch.float64, device=x.device)
    _check(lib().sba_block_means(_ptr(x), B, H, Npad, D, _ptr(_valid_len(valid_len, x.device)), block,
                                 _ptr(out), _stream(stream)), "sba_block_means")
    return out


def attention(q, k, v, kv_idx, kv_cnt, valid_len=None, softmax_scale: float = 0.0, out=None,
              lse=None, want_lse: bool = True, block: int = BLOCK, stream=None):
    """Block-sparse attention under a routing.  Returns (o bf16, lse fp32 or None)."""
    B, H, Npad, D = _qkv(q, k, v)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, H, Npad), dtype=torch.float32, device=q.device)
    if not (kv_idx.dtype == torch.int32 and kv_cnt.dtype == torch.int32 and kv_idx.is_contiguous()
            and kv_cnt.is_contiguous() and kv_idx.is_cuda and kv_cnt.is_cuda):
        raise ValueError("kv_idx / kv_cnt must be contiguous int32 CUDA tensors")
    _check(lib().sba_attention(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Npad, D,
                               _ptr(_valid_len(valid_len, q.device)), block, _ptr(kv_idx),
                               _ptr(kv_cnt), kv_idx.shape[-1], float(softmax_scale), _stream(stream)),
           "sba_attention")
    return out, lse


def pair_query_blocks(kv_idx, kv_cnt, valid_len=None, block: int = BLOCK, pair_order=None,
                      workspace=None, stream=None):
    """Tiles of two query blocks with overlapping kept lists: int32 [B, H, 2*ceil(nQ/2)]."""
    B, H, nQ, kmax = kv_idx.shape
    Npad = nQ * block
    if pair_order is None:
        pair_order = torch.empty((B, H, 2 * ((nQ + 1) // 2)), dtype=torch.int32, device=kv_idx.device)
    if workspace is None:
        workspace = torch.empty(int(lib().sba_pair_workspace_size(B, H, Npad, block)), dtype=torch.uint8,
                                device=kv_idx.device)
    _check(lib().sba_pair_query_blocks(_ptr(kv_idx), _ptr(kv_cnt), B, H, Npad, kmax,
                                       _ptr(_valid_len(valid_len, kv_idx.device)), block, _ptr(pair_order),
                                       _ptr(workspace), workspace.numel(), _stream(stream)),
           "sba_pair_query_blocks")
    return pair_order


def attention_paired(q, k, v, kv_idx, kv_cnt, pair_order, valid_len=None, softmax_scale: float = 0.0,
                     out=None, lse=None, want_lse: bool = True, block: int = BLOCK, stream=None):
    """sba_attention over the tiles of `pair_order`.  Returns (o bf16, lse fp32 or None)."""
    B, H, Npad, D = _qkv(q, k, v)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, H, Npad), dtype=torch.float32, device=q.device)
    _check(lib().sba_attention_paired(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Npad, D,
                                      _ptr(_valid_len(valid_len, q.device)), block, _ptr(kv_idx),
                                      _ptr(kv_cnt), kv_idx.shape[-1], _ptr(pair_order), float(softmax_scale),
                                      _stream(stream)), "sba_attention_paired")
    return out, lse


def attention_to_shards(q, k, v, kv_idx, kv_cnt, o_shards, lse_shards=None, h_first: int = 0, h_total=None,
                        valid_len=None, pair_order=None, softmax_scale: float = 0.0, block: int = BLOCK,
                        stream=None):
    """Attention for this caller's heads h_first .. h_first + H - 1 (q, k, v: [B, H, Npad, D],
    the whole sequence), each output row stored straight into the sequence shard that owns
    its token: o_shards[s] is bf16 [B, h_total, Npad / len(o_shards), D] (a tensor, or a raw
    device pointer such as a peer's symmetric-memory buffer, then h_total is required);
    lse_shards likewise fp32 [B, h_total, Npad / len(o_shards)] or None."""
    B, H, Npad, D = _qkv(q, k, v)
    n = len(o_shards)
    if n < 1 or n > 8:
        raise ValueError("between 1 and 8 output shards")
    ptr = lambda t: int(t) if isinstance(t, int) else t.data_ptr()
    if h_total is None:
        if isinstance(o_shards[0], int):
            raise ValueError("h_total is required with raw shard pointers")
        h_total = o_shards[0].shape[1]
    for t in list(o_shards) + list(lse_shards or []):
        if not isinstance(t, int):
            exp = torch.bfloat16 if t.dim() == 4 else torch.float32
            shape = (B, h_total, Npad // n) + ((D,) if t.dim() == 4 else ())
            if t.dtype != exp or tuple(t.shape) != shape or not t.is_contiguous() or t.device != q.device:
                raise ValueError(f"shard of shape {tuple(t.shape)} / {t.dtype}; expected {shape} / {exp}, contiguous")
    o_arr = (ctypes.c_void_p * n)(*[ptr(t) for t in o_shards])
    l_arr = None if lse_shards is None else (ctypes.c_void_p * n)(*[ptr(t) for t in lse_shards])
    _check(lib().sba_attention_to_shards(_ptr(q), _ptr(k), _ptr(v), ctypes.cast(o_arr, ctypes.c_void_p),
                                         None if l_arr is None else ctypes.cast(l_arr, ctypes.c_void_p), n,
                                         int(h_total), int(h_first), B, H, Npad, D,
                                         _ptr(_valid_len(valid_len, q.device)), block, _ptr(kv_idx), _ptr(kv_cnt),
                                         kv_idx.shape[-1], _ptr(pair_order), float(softmax_scale), _stream(stream)),
           "sba_attention_to_shards")


def attention_compensated(q, k, v, kv_idx, kv_cnt, valid_len=None, pair_order=None, softmax_scale: float = 0.0,
                          out=None, lse=None, want_lse: bool = True, block: int = BLOCK, stream=None):
    """Block-sparse attention with the dropped blocks compensated to first order about
    their mean keys (see include/sba.h).  Returns (o bf16, lse fp32 or None)."""
    B, H, Npad, D = _qkv(q, k, v)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, H, Npad), dtype=torch.float32, device=q.device)
    _check(lib().sba_attention_compensated(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Npad, D,
                                           _ptr(_valid_len(valid_len, q.device)), block, _ptr(kv_idx), _ptr(kv_cnt),
                                           kv_idx.shape[-1], _ptr(pair_order), float(softmax_scale),
                                           _stream(stream)), "sba_attention_compensated")
    return out, lse


def mean_compensation_workspace_size(B: int, H: int, Npad: int, D: int, block: int = BLOCK) -> int:
    return int(lib().sba_mean_compensation_workspace_size(B, H, Npad, D, block))


def attention_mean_compensated(q, k, v, kv_idx, kv_cnt, valid_len=None, pair_order=None, softmax_scale: float = 0.0,
                               out=None, lse=None, want_lse: bool = True, workspace=None, block: int = BLOCK,
                               stream=None):
    """Block-sparse attention with each dropped block as one softmax entry carrying its
    mean key and value (the zeroth-order form; see include/sba.h).  Returns (o, lse)."""
    B, H, Npad, D = _qkv(q, k, v)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, H, Npad), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(mean_compensation_workspace_size(B, H, Npad, D, block), dtype=torch.uint8,
                                device=q.device)
    _check(lib().sba_attention_mean_compensated(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Npad, D,
                                                _ptr(_valid_len(valid_len, q.device)), block, _ptr(kv_idx),
                                                _ptr(kv_cnt), kv_idx.shape[-1], _ptr(pair_order),
                                                float(softmax_scale), _ptr(workspace), workspace.numel(),
                                                _stream(stream)), "sba_attention_mean_compensated")
    return out, lse


def dense_attention(q, k, v, valid_len=None, softmax_scale: float = 0.0, out=None, lse=None,
                    want_lse: bool = True, stream=None):
    """Dense attention over each sample's valid tokens.  Returns (o bf16, lse fp32 or None)."""
    B, H, Npad, D = _qkv(q, k, v)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, H, Npad), dtype=torch.float32, device=q.device)
    _check(lib().sba_dense_attention(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Npad, D,
                                     _ptr(_valid_len(valid_len, q.device)), float(softmax_scale),
                                     _stream(stream)), "sba_dense_attention")
    return out, lse


def sparse_attention(q, k, v, valid_len=None, sparsity: float = 0.75, softmax_scale: float = 0.0,
                     router: str = "mean", budget: int = 1, stream=None):
    """The whole path: routing, tile pairing, block-sparse attention.
    router "mean": block-mean scores (sba_pool_select); "lse": sub-block
    log-sum-exp scores with an optional kept-count budget (sba_pool_select_lse).
    Returns (o, lse, kv_idx, kv_cnt)."""
    if router == "mean":
        kv_idx, kv_cnt = pool_select(q, k, valid_len, sparsity, stream=stream)
    elif router == "lse":
        kv_idx, kv_cnt = pool_select_lse(q, k, valid_len, sparsity, budget=budget, stream=stream)
    else:
        raise ValueError(f"unknown router {router!r}")
    pair_order = pair_query_blocks(kv_idx, kv_cnt, valid_len, stream=stream)
    o, lse = attention_paired(q, k, v, kv_idx, kv_cnt, pair_order, valid_len, softmax_scale, stream=stream)
    return o, lse, kv_idx, kv_cnt


def keep_token_count(n_tokens: int, ratio: float) -> int:
    """Tokens saliency pruning keeps of n: clamp(ceil(ratio * n - 1e-9), 1, n)."""
    return int(lib().sba_keep_token_count(int(n_tokens), float(ratio)))


def token_prune(x, valid_len=None, ratio: float = 0.5, npad_out: int | None = None, idx=None, valid_out=None,
                workspace=None, stream=None):
    """Token pruning by feature-norm saliency (see include/sba.h).  x: bf16 [B, N, C]
    token features.  Returns (idx int32 [B, npad_out]: the kept tokens' indices in
    their original order, then -1; valid_out int32 [B]: the kept counts).  npad_out
    defaults to the kept count of a full sample rounded up to a multiple of 64."""
    if not (x.is_cuda and x.dtype == torch.bfloat16 and x.dim() == 3 and x.is_contiguous()):
        raise ValueError("expected a contiguous bf16 CUDA tensor [B, N, C]")
    B, N, C = x.shape
    if npad_out is None:
        npad_out = -(-keep_token_count(N, ratio) // BLOCK) * BLOCK
    if idx is None:
        idx = torch.empty((B, npad_out), dtype=torch.int32, device=x.device)
    if valid_out is None:
        valid_out = torch.empty((B,), dtype=torch.int32, device=x.device)
    if workspace is None:
        workspace = torch.empty(int(lib().sba_token_prune_workspace_size(B, N)), dtype=torch.uint8,
                                device=x.device)
    _check(lib().sba_token_prune_select(_ptr(x), B, N, C, _ptr(_valid_len(valid_len, x.device)), float(ratio),
                                        int(npad_out), _ptr(idx), _ptr(valid_out), _ptr(workspace),
                                        workspace.numel(), _stream(stream)), "sba_token_prune_select")
    return idx, valid_out


def gather_tokens(src, idx, valid_out, out=None, stream=None):
    """The kept rows of a per-token tensor, compacted: src [B, H, N, ...] or [B, N, ...]
    (any dtype, a row of 4k bytes), idx / valid_out as token_prune returns them.  Rows
    past a sample's kept count are zero.  Returns [B, H, npad_out, ...] / [B, npad_out, ...]."""
    if not (src.is_cuda and src.is_contiguous() and src.dim() >= 3):
        raise ValueError("expected a contiguous CUDA tensor [B, H, N, ...] or [B, N, ...]")
    B, npad_out = idx.shape
    heads = src.dim() == 4
    H, N = (src.shape[1], src.shape[2]) if heads else (1, src.shape[1])
    rest = src.shape[3:] if heads else src.shape[2:]
    row_bytes = src.element_size() * math.prod(rest)
    shape = (B, H, npad_out, *rest) if heads else (B, npad_out, *rest)
    if out is None:
        out = torch.empty(shape, dtype=src.dtype, device=src.device)
    _check(lib().sba_gather_tokens(_ptr(src), B, H, N, row_bytes, _ptr(idx), _ptr(valid_out), int(npad_out),
                                   _ptr(out), _stream(stream)), "sba_gather_tokens")
    return out


# ---------------------------------------------------------------- the block around the attention
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_NORMS = {None: 0, "layer": 1, "rms": 2}
_ACTS = {None: 0, "gelu_tanh": 1, "silu": 2}
_LAYOUTS = {"interleaved": 0, "half": 1}
_Strides3, _Strides5, _Strides6, _Strides8 = (ctypes.c_int64 * n for n in (3, 5, 6, 8))


def _elsewhere(device, stream):
    """The context of a call on GPU `device` (its index): allocations and launch on `stream`, or
    on the device's current stream.  None when that is where the caller is already."""
    if device < 0:
        raise ValueError("expected CUDA tensors")
    if stream is None:
        return None if device == torch._C._cuda_getDevice() else torch.cuda.device(device)
    if stream.device.index != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{device}")
    return torch.cuda.stream(stream)


def _counts(*sizes):
    """Refuse sizes that do not fit the C calls' 32-bit arguments (ctypes would cut them)."""
    if max(sizes) > 0x7fffffff:
        raise ValueError(f"sizes {sizes}: each must be below 2^31")


def _values(t, name, shape, device, dtype):
    """Check an optional tensor: shape, device, type, contiguous."""
    if t is not None and not (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device):
        raise ValueError(f"{name}: expected a contiguous {tuple(shape)} tensor of {dtype} on cuda:{device}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")


def _rows(t, name, shape, device, dtype, written=False):
    """Check rows at any strides: the last dimension contiguous, and no two elements of a
    written tensor in one place."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype} on cuda:{device}, got {tuple(t.shape)} {t.dtype} on "
                         f"{t.device}")
    if t.is_contiguous():
        return
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if written:
        reach = 0
        for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1):
            if stride <= reach:
                raise ValueError(f"{name}: written elements overlap")
            reach += stride * (size - 1)


def _params(params, shape, dtype, device, kind=None):
    """Check parameters (name, tensor or None) of one shape and one type, fp32 or `dtype`: that
    of `kind`, where earlier ones have set it.  Returns the type, or None as it came."""
    for name, t in params:
        if t is None:
            continue
        if kind is None:
            kind = t.dtype
            if kind != torch.float32 and kind != dtype:
                raise ValueError(f"{name}: expected torch.float32 or {dtype}, got {kind}")
        _values(t, name, shape, device, kind)
    return kind


def _tables(tables, C, index, rows, dtype, device, kind=None):
    """Check modulation tables [G, C] (name, tensor or None) and the index of their rows;
    without an index sample b takes row b, so G = B.  Returns (G, the parameters' type)."""
    G = 0
    for _, t in tables:
        if t is not None:
            G = t.shape[0] if t.dim() == 2 else 0
            if not G:
                raise ValueError("gate, scale and shift must be [G, C], G at least 1")
            break
    if index is not None:
        if not G:
            raise ValueError("an index, and nothing that it selects from")
        _values(index, "index", rows, device, torch.int32)
    elif G and G != (rows[0] if len(rows) == 2 else 1):
        raise ValueError(f"{G} modulation rows for a batch of {rows[0] if len(rows) == 2 else 1}, and no index")
    return G, _params(tables, (G, C), dtype, device, kind)


def residual_norm(x, y=None, gate=None, norm="layer", weight=None, bias=None, scale=None, shift=None, index=None,
                  post_norm=None, post_weight=None, valid_len=None, eps: float = 1e-6, quantize: bool = False,
                  out_dtype=None, x_out=None, out=None, out_scale=None, stream=None):
    """The gated residual of a block's output y, and the modulated norm of the new residual
    stream, in one pass (see include/sba.h).

      r = x + gate * post_norm(y) * post_weight
      h = (norm(r) * weight + bias) * (1 + scale) + shift

    x: [B, N, C] bf16, fp16 or fp32; y the same type, or 16-bit next to an fp32 x; both at
    any strides with contiguous rows.  norm, post_norm: "layer", "rms" or None.  weight,
    bias, post_weight: [C]; gate, scale, shift: [G, C], row b for sample b, or row
    index[b, n] with an int32 index [B, N]; all fp32 or of h's type.  Rows past
    valid_len[b] come out as zeros.

    Returns (r, h); r is x itself when there is no y, h is None with norm=None.  With
    quantize=True returns (r, codes, scales) for int8_linear: int8 [B, N, C rounded up to
    16] and fp32 [B, N].  h has y's type (out_dtype without a y, x's by default).  x_out
    may be x, out may be y."""
    where = _elsewhere(x.get_device(), stream)
    if where is not None:
        with where:
            return residual_norm(x, y, gate, norm, weight, bias, scale, shift, index, post_norm, post_weight, valid_len,
                                 eps, quantize, out_dtype, x_out, out, out_scale)
    shape, dev, xtype = x.shape, x.get_device(), x.dtype
    if len(shape) != 3 or xtype not in _DTYPES:
        raise ValueError("x: expected [B, N, C] in bf16, fp16 or fp32")
    B, N, C = shape
    dtype = y.dtype if y is not None else (out_dtype or xtype)
    if dtype not in _DTYPES or (dtype != xtype and xtype != torch.float32) or (
            out_dtype is not None and out_dtype != dtype):
        raise ValueError(f"x of {xtype}, y of {None if y is None else y.dtype}, out_dtype {out_dtype}: h has y's "
                         "type, and that is x's or, next to an fp32 x, 16-bit")
    if norm not in _NORMS or post_norm not in _NORMS:
        raise ValueError(f"norm {norm!r}, post_norm {post_norm!r}: each one of {sorted(map(str, _NORMS))}")
    if norm is None and (quantize or y is None):
        raise ValueError("norm=None needs a y, and gives nothing to quantize")
    _rows(x, "x", shape, dev, xtype)
    ptype = None
    if weight is not None or bias is not None or post_weight is not None:
        ptype = _params((("weight", weight), ("bias", bias), ("post_weight", post_weight)), (C,), dtype, dev)
    G = 0
    if gate is not None or scale is not None or shift is not None or index is not None:
        G, ptype = _tables((("gate", gate), ("scale", scale), ("shift", shift)), C, index, (B, N), dtype, dev, ptype)
    if valid_len is not None:
        _values(valid_len, "valid_len", (B,), dev, torch.int32)
    strides = [x.stride(0), x.stride(1), 0, 0, 0, 0, 0, 0]
    if y is not None:
        _rows(y, "y", shape, dev, dtype)
        if x_out is None:
            x_out = x.new_empty(shape)
        else:
            _rows(x_out, "x_out", shape, dev, xtype, written=True)
        strides[2:6] = y.stride(0), y.stride(1), x_out.stride(0), x_out.stride(1)
    elif x_out is not None:
        raise ValueError("x_out without a y: the residual stream does not change")
    if norm is not None:
        if quantize:
            shape, kind = (B, N, -(-C // 16) * 16), torch.int8
            if out_scale is None:
                out_scale = x.new_empty((B, N), dtype=torch.float32)
            else:
                _values(out_scale, "out_scale", (B, N), dev, torch.float32)
        else:
            kind = dtype
        if out is None:
            out = x.new_empty(shape, dtype=kind)
        else:
            _rows(out, "out", shape, dev, kind, written=True)
        strides[6:8] = out.stride(0), out.stride(1)
    elif out is not None:
        raise ValueError("out without a norm")
    if out_scale is not None and not quantize:
        raise ValueError("out_scale without quantize")
    if B and N:
        _counts(B, N, C)
        _check(lib().sba_residual_norm(
            x.data_ptr(), _raw(y), _raw(x_out), _raw(out), _raw(out_scale), _DTYPES[xtype], _DTYPES[dtype], B, N, C,
            _Strides8(*strides), _raw(valid_len), _NORMS[norm], _raw(weight), _raw(bias), _NORMS[post_norm],
            _raw(post_weight), _raw(gate), _raw(scale), _raw(shift), 2 if ptype is None else _DTYPES[ptype], G,
            _raw(index), eps, torch._C._cuda_getCurrentRawStream(dev)), "sba_residual_norm")
    r = x if y is None else x_out
    return (r, out, out_scale) if quantize else (r, out)


def token_quantize(x, codes=None, scales=None, stream=None):
    """Rows in 8 bits with one scale a row: scales = max|row| / 127, codes the nearest integers
    (see include/sba.h).  x: [..., K] of bf16, fp16 or fp32, [M, K] (tokens, or a weight's
    output channels), [B, N, K], or the attention's head layout [B, H, N, D], whose K = H * D;
    at any strides with contiguous rows.  Returns (codes int8 [M, K'] or [B, N, K'], scales
    fp32 [M] or [B, N]), K' = K rounded up to a multiple of 16 (zero codes)."""
    dev = x.get_device()
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return token_quantize(x, codes, scales)
    shape, strides = x.shape, x.stride()
    kind = _DTYPES.get(x.dtype)
    if kind is None or not 2 <= len(shape) <= 4 or (strides[-1] != 1 and shape[-1] > 1):
        raise ValueError("x: expected [M, K], [B, N, K] or [B, H, N, D] in bf16, fp16 or fp32, its last dimension "
                         "contiguous")
    if len(shape) == 4:
        (B, H, N, D), (sb, sh, sn, _) = shape, strides
        lead = (B, N)
    elif len(shape) == 3:
        (B, N, D), (sb, sn, _), H, sh = shape, strides, 1, 0
        lead = (B, N)
    else:
        (N, D), (sn, _), B, H, sb, sh = shape, strides, 1, 1, 0, 0
        lead = (N,)
    width = -(-(H * D) // 16) * 16
    if codes is None:
        codes = x.new_empty((*lead, width), dtype=torch.int8)
    else:
        _values(codes, "codes", (*lead, width), dev, torch.int8)
    if scales is None:
        scales = x.new_empty(lead, dtype=torch.float32)
    else:
        _values(scales, "scales", lead, dev, torch.float32)
    if B and N:
        _counts(B, H, N, D)
        _check(lib().sba_token_quantize(x.data_ptr(), kind, B, H, N, D, _Strides3(sb, sh, sn), codes.data_ptr(),
                                        scales.data_ptr(), torch._C._cuda_getCurrentRawStream(dev)), "sba_token_quantize")
    return codes, scales


def int8_linear(codes, scales, weight_codes, weight_scales, bias=None, activation=None, gate=None, index=None,
                residual=None, out_dtype=torch.bfloat16, heads=None, out=None, stream=None):
    """A projection in 8-bit integers with its epilogue (see include/sba.h):

      out = residual + gate * activation((codes @ weight_codes.T) * scales * weight_scales + bias)

    codes int8 [N, K] or [B, N, K] and scales fp32 [N] or [B, N] as residual_norm and
    token_quantize give them; weight_codes int8 [M, K] and weight_scales fp32 [M]
    (token_quantize of the weight).  activation: None, "gelu_tanh" or "silu".  bias: [M];
    gate: [G, M], row b for sample b or row index[b, n]; both fp32 or of out's type.
    residual: of out's shape and type, contiguous rows, may be out.  Returns out [..., M]; with
    heads=H (and codes [B, N, K]) the attention's layout [B, H, N, M / H] instead."""
    shape, dev = codes.shape, codes.get_device()
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return int8_linear(codes, scales, weight_codes, weight_scales, bias, activation, gate, index, residual,
                               out_dtype, heads, out)
    if len(shape) == 3:
        B, N, K = shape
        lead = (B, N)
    elif len(shape) == 2:
        (N, K), B = shape, 1
        lead = (N,)
    else:
        raise ValueError("codes: expected [N, K] or [B, N, K]")
    if weight_codes.dim() != 2:
        raise ValueError("weight_codes: expected [M, K]")
    M = weight_codes.shape[0]
    _values(codes, "codes", shape, dev, torch.int8)
    _values(scales, "scales", lead, dev, torch.float32)
    _values(weight_codes, "weight_codes", (M, K), dev, torch.int8)
    _values(weight_scales, "weight_scales", (M,), dev, torch.float32)
    otype = _DTYPES.get(out_dtype)
    if otype is None:
        raise ValueError(f"out_dtype {out_dtype}: expected bf16, fp16 or fp32")
    if activation not in _ACTS:
        raise ValueError(f"unknown activation {activation!r}; one of {sorted(map(str, _ACTS))}")
    if heads is not None and (len(lead) != 2 or heads < 1 or M % heads or residual is not None):
        raise ValueError("heads: codes [B, N, K], a divisor of M, and no residual")
    ptype, G = None, 0
    if bias is not None:
        ptype = _params((("bias", bias),), (M,), out_dtype, dev)
    if gate is not None or index is not None:
        G, ptype = _tables((("gate", gate),), M, index, lead, out_dtype, dev, ptype)
    shape = (B, heads, N, M // heads) if heads else (*lead, M)
    if out is None:
        out = codes.new_empty(shape, dtype=out_dtype)
    else:
        _rows(out, "out", shape, dev, out_dtype, written=True)
    rb = rn = 0
    if residual is not None:
        _rows(residual, "residual", shape, dev, out_dtype)
        rb, rn = residual.stride()[:2] if len(lead) == 2 else (0, residual.stride(0))
    strides = out.stride()
    ob, oh, on = strides[:3] if heads else (strides[0], 0, strides[1]) if len(lead) == 2 else (0, 0, strides[0])
    if B and N:
        _counts(B, N, K, M)
        _check(lib().sba_int8_linear(
            codes.data_ptr(), scales.data_ptr(), weight_codes.data_ptr(), weight_scales.data_ptr(), B, N, K, M,
            _raw(bias), _raw(gate), 2 if ptype is None else _DTYPES[ptype], G, _raw(index), _ACTS[activation],
            _raw(residual), out.data_ptr(), otype, heads or 0, _Strides5(rb, rn, ob, oh, on),
            torch._C._cuda_getCurrentRawStream(dev)), "sba_int8_linear")
    return out


class RopeTable:
    """The frequencies of `rotary`: radians a position and the position axis of each of
    rope_dim / 2 channel pairs, and the factor on the turned channels."""

    def __init__(self, inv_freq, axis=None, amplitude: float = 1.0):
        self.inv_freq = tuple(float(f) for f in inv_freq)
        self.axis = tuple(int(a) for a in axis) if axis is not None else (0,) * len(self.inv_freq)
        self.amplitude = float(amplitude)
        n = len(self.inv_freq)
        if n == 0 or len(self.axis) != n or min(self.axis) < 0 or max(self.axis) > 254:
            raise ValueError("one axis in 0..254 for each pair's frequency, and a pair at least")
        if not all(math.isfinite(f) for f in self.inv_freq) or not math.isfinite(self.amplitude):
            raise ValueError("frequencies and amplitude must be finite")
        self.rope_dim = 2 * n
        self.axes = max(self.axis) + 1
        self._freq = (ctypes.c_double * n)(*self.inv_freq)
        self._axis = (ctypes.c_uint8 * n)(*self.axis)
        self._freq_at, self._axis_at = ctypes.addressof(self._freq), ctypes.addressof(self._axis)

    def __reduce__(self):
        # a copy makes its own arrays: the addresses are of this table's
        return RopeTable, (self.inv_freq, self.axis, self.amplitude)


def rope_frequencies(rope_dim: int, axes: int = 1, base: float = 10000.0, scaling=None, factor: float = 1.0,
                     original_length: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0) -> RopeTable:
    """The usual frequencies base^(-2i/d) of rope_dim channels split evenly into `axes` axes
    of d channels each, for positions past the trained length scaled by `factor`:

      None      as they are
      "linear"  every frequency / factor
      "ntk"     base * factor^(d / (d - 2)) in place of base
      "yarn"    pairs that turn at least beta_fast times within original_length positions as
                they are, those that turn at most beta_slow times / factor, a linear ramp over
                the pairs between; amplitude 0.1 ln(factor) + 1"""
    if axes < 1 or rope_dim < 2 or rope_dim % (2 * axes):
        raise ValueError("rope_dim must split into an even number of channels an axis")
    if not (base > 0 and math.isfinite(base) and factor > 0 and math.isfinite(factor)):
        raise ValueError("base and factor must be positive and finite")
    d = rope_dim // axes
    amplitude = 1.0
    if scaling == "ntk":
        if d == 2:
            raise ValueError("ntk scaling needs more than one pair an axis")
        base = base * factor ** (d / (d - 2))
    freq = [base ** (-2.0 * i / d) for i in range(d // 2)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "yarn":
        if base <= 1 or original_length < 1 or not 0 < beta_slow < beta_fast:
            raise ValueError("yarn scaling: base > 1, original_length >= 1 and 0 < beta_slow < beta_fast")
        # the pair index that turns `turns` times within the original length
        pair = lambda turns: d * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))
        slow = pair(beta_slow)
        lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(slow), d - 1)
        # (no pair turns beta_slow times within a short length: then lo = hi = 0, and no ramp)
        ramp = [1.0 if i >= slow else min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(d // 2)]
        freq = [f / factor * t + f * (1 - t) for f, t in zip(freq, ramp)]
        amplitude = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return RopeTable(freq * axes, [a for a in range(axes) for _ in range(d // 2)], amplitude)


def rotary(x, pos, table: RopeTable, layout: str = "interleaved", inverse: bool = False, out=None, stream=None):
    """Rotary positions (see include/sba.h): the first table.rope_dim channels of x [B, H, N, D]
    turned by the token's position, the others copied.  x: bf16, fp16 or fp32 at any strides
    with contiguous channels (a token-major [B, N, H, D] tensor is x.transpose(1, 2)).  pos:
    int32 [B, N, table.axes], or [B, N] for one axis.  layout: pairs of channels (2p, 2p + 1),
    "interleaved", or (p, p + rope_dim / 2), "half".  inverse turns back, which is also the
    gradient.  out may be x.  Returns out (laid out as x)."""
    shape, dev, strides = x.shape, x.get_device(), x.stride()
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return rotary(x, pos, table, layout, inverse, out)
    dtype = _DTYPES.get(x.dtype)
    if len(shape) != 4 or dtype is None:
        raise ValueError("x: expected [B, H, N, D] in bf16, fp16 or fp32")
    B, H, N, D = shape
    if layout not in _LAYOUTS:
        raise ValueError(f"unknown layout {layout!r}; one of {sorted(_LAYOUTS)}")
    if table.rope_dim > D:
        raise ValueError(f"a table of {table.rope_dim} channels for heads of {D}")
    _rows(x, "x", shape, dev, x.dtype)
    _values(pos, "pos", (B, N) if pos.dim() == 2 and table.axes == 1 else (B, N, table.axes), dev, torch.int32)
    if out is None:
        out = torch.empty_like(x)  # of an expanded x: dense
    else:
        _rows(out, "out", shape, dev, x.dtype, written=True)
        if out.data_ptr() == x.data_ptr() and out.stride() != strides:
            raise ValueError("out at x's place with other strides")
    if B and H and N:
        _counts(B, H, N, D)
        _check(lib().sba_rotary(x.data_ptr(), out.data_ptr(), dtype, pos.data_ptr(), table.axes, B, H, N, D,
                                _Strides6(*strides[:3], *out.stride()[:3]), table.rope_dim, _LAYOUTS[layout],
                                table._freq_at, table._axis_at, table.amplitude, int(inverse),
                                torch._C._cuda_getCurrentRawStream(dev)), "sba_rotary")
    return out


def device_status(stream=None) -> int:
    """Synchronise the stream; return and clear the device-side error word (an SBA_* code)."""
    return int(lib().sba_get_device_status(_stream(stream)))


def set_wait_limit(cycles: int) -> None:
    lib().sba_set_wait_limit(int(cycles))


_ATTN_KERNELS = {"auto": 0, "query_pairs": 1, "cta_pair": 2}


def set_attention_kernel(which: str) -> None:
    """Which D = 128 attention kernel the attention calls run (process-wide):
    "query_pairs" (one SM per two query blocks), "cta_pair" (a 2-SM cluster per four
    query blocks) or "auto" (the query pairs, the faster one on B200)."""
    if which not in _ATTN_KERNELS:
        raise ValueError(f"unknown attention kernel {which!r}; one of {sorted(_ATTN_KERNELS)}")
    _check(lib().sba_set_attention_kernel(_ATTN_KERNELS[which]), "sba_set_attention_kernel")
