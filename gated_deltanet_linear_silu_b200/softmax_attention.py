"""The softmax-attention layers between the linear ones, for serving: q/k norm
with the rotation, the paged key/value cache and the attention of drafted
tokens over it. Argument marshalling over the C ABI (include/gdn.h), like the
rest of the package.

A decode step of such a layer:

    q = qk_norm_rope_cache(q, k, v, q_w, k_w, positions, inv_freq, cache, page_table, seq_lens, cu_seqlens)
    o = tree_attention(q, cache, page_table, seq_lens, cu_seqlens, mask=mask, max_nodes=nodes, gate=gate)
    seq_lens = kv_cache_accept(cache, page_table, seq_lens, cu_seqlens, accepted)   # after verification
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Tuple

import torch

from . import _check, _cuda, _dtype_code, _on, _ptr, _stream, _token_stride, lib

GDN_BF16, GDN_E4M3 = 1, 2


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page", ctypes.c_int),
                ("Hk", ctypes.c_int), ("D", ctypes.c_int), ("dtype", ctypes.c_int)]


class KVCache(NamedTuple):
    """Pages of one layer's keys and values: k, v [n_pages, Hk, page, D] in
    bf16, or in e4m3 with fp32 scales k_scale, v_scale [n_pages, Hk, page]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None


def kv_cache(n_pages: int, page: int, Hk: int, D: int, *, dtype: torch.dtype = torch.float8_e4m3fn,
             device=None) -> KVCache:
    """An empty (zero) cache of n_pages pages of `page` tokens."""
    if dtype not in (torch.float8_e4m3fn, torch.bfloat16):
        raise TypeError(f"unsupported cache dtype {dtype} (float8_e4m3fn or bfloat16)")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    k, v = (torch.zeros((n_pages, Hk, page, D), dtype=dtype, device=device) for _ in range(2))
    if dtype == torch.bfloat16:
        return KVCache(k, v)
    ks, vs = (torch.zeros((n_pages, Hk, page), dtype=torch.float32, device=device) for _ in range(2))
    return KVCache(k, v, ks, vs)


def rope_inv_freq(rotary: int, base: float = 1e7, device=None) -> torch.Tensor:
    """Radians per position of each rotated pair: base^(-2i / rotary), fp64."""
    return float(base) ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=device) / rotary)


def tree_mask(parents: torch.Tensor, cu_seqlens: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """(mask int64 [T], depth int32 [T]) of drafted trees: parents [T] int holds
    each node's parent as a number within its sequence, below its own (-1: the
    node follows the context directly). Bit j of a node's mask is set for
    itself and its ancestors; its depth is the number of ancestors, so that its
    position is seq_len - nodes + depth."""
    par, cu = parents.tolist(), cu_seqlens.tolist()
    mask, depth = [0] * len(par), [0] * len(par)
    for a, b in zip(cu, cu[1:]):
        if not 0 <= a <= b <= len(par) or b - a > 64:
            raise ValueError("cu_seqlens does not fit parents, or a sequence has more than 64 nodes")
        for t in range(a, b):
            p = int(par[t])
            if not -1 <= p < t - a:
                raise ValueError(f"parent {p} of node {t - a}: a parent comes before its children")
            mask[t] = (1 << (t - a)) | (mask[a + p] if p >= 0 else 0)
            depth[t] = depth[a + p] + 1 if p >= 0 else 0
    signed = [m - (1 << 64) if m >> 63 else m for m in mask]
    dev = parents.device
    return (torch.tensor(signed, dtype=torch.int64, device=dev), torch.tensor(depth, dtype=torch.int32, device=dev))


def _cache_arg(cache: KVCache) -> _CacheStruct:
    k, v, ks, vs = cache
    if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("the cache's k and v must be [n_pages, Hk, page, D] alike")
    if k.dtype == torch.float8_e4m3fn:
        if ks is None or vs is None or ks.shape != k.shape[:3] or vs.shape != k.shape[:3]:
            raise ValueError("an e4m3 cache needs k_scale and v_scale [n_pages, Hk, page]")
        if ks.dtype != torch.float32 or vs.dtype != torch.float32:
            raise TypeError("the cache's scales must be fp32")
        code = GDN_E4M3
    elif k.dtype == torch.bfloat16:
        code, ks, vs = GDN_BF16, None, None
    else:
        raise TypeError(f"unsupported cache dtype {k.dtype} (float8_e4m3fn or bfloat16)")
    _cuda(k, v, ks, vs)
    P, Hk, page, D = k.shape
    at = lambda t: None if t is None else t.data_ptr()
    return _CacheStruct(at(k), at(v), at(ks), at(vs), P, page, Hk, D, code)


def _pages(page_table: torch.Tensor, seq_lens: torch.Tensor, cu_seqlens: torch.Tensor):
    """Checked (page_table, max_pages, seq_lens, cu_seqlens, N) arguments."""
    for name, t in (("page_table", page_table), ("seq_lens", seq_lens), ("cu_seqlens", cu_seqlens)):
        if t.dtype != torch.int32:
            raise TypeError(f"{name} must be int32")
    N = cu_seqlens.shape[0] - 1
    if cu_seqlens.dim() != 1 or N < 0 or tuple(seq_lens.shape) != (N,) or page_table.dim() != 2 \
            or page_table.shape[0] != N:
        raise ValueError("page_table must be [N, max_pages], seq_lens [N] and cu_seqlens [N + 1]")
    _cuda(page_table, seq_lens, cu_seqlens)
    return _ptr(page_table), page_table.shape[1], _ptr(seq_lens), _ptr(cu_seqlens), N


def _same_device(dev: torch.device, *ts):
    for t in ts:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors must be on one device: {t.device} and {dev}")


def _norm_args(q, k, q_w, k_w, positions, inv_freq):
    T, H, D = q.shape
    if k.dim() != 3 or k.shape[0] != T or k.shape[2] != D or k.dtype != q.dtype:
        raise ValueError("q must be [T, H, D] and k [T, Hk, D] of one dtype")
    if tuple(q_w.shape) != (D,) or tuple(k_w.shape) != (D,) or q_w.dtype != torch.float32 \
            or k_w.dtype != torch.float32:
        raise ValueError("q_w and k_w must be [D] fp32")
    if tuple(positions.shape) != (T,) or positions.dtype != torch.int32:
        raise ValueError("positions must be [T] int32")
    if inv_freq.dim() != 1 or inv_freq.dtype != torch.float64 or 2 * inv_freq.shape[0] > D:
        raise ValueError("inv_freq must be [rotary / 2] fp64, rotary at most D")
    _cuda(q_w, k_w, positions, inv_freq)
    _same_device(q.device, k, q_w, k_w, positions, inv_freq)
    return T, H, D, 2 * inv_freq.shape[0]


def _out(given: Optional[torch.Tensor], shape, dtype, device) -> torch.Tensor:
    if given is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(given.shape) != tuple(shape) or given.dtype != dtype or given.device != device:
        raise ValueError(f"an output must be {tuple(shape)} {dtype} on {device}")
    _cuda(given)
    return given


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_w: torch.Tensor, k_w: torch.Tensor, positions: torch.Tensor,
                 inv_freq: torch.Tensor, *, eps: float = 1e-6, interleaved: bool = False,
                 out_q: Optional[torch.Tensor] = None, out_k: Optional[torch.Tensor] = None
                 ) -> Tuple[torch.Tensor, torch.Tensor]:
    """RMSNorm of each head of q [T, H, D] and k [T, Hk, D] (bf16 or fp32; either
    may be a token-strided view, e.g. of the fused projection), times q_w, k_w
    [D] fp32, and the rotation of the first 2 * len(inv_freq) elements by
    positions [T] int32 (inv_freq fp64, see rope_inv_freq; pairs are the two
    halves, or neighbours when interleaved). Returns (q, k), dense; out_q, out_k
    may be the inputs themselves where those are dense."""
    T, H, D, rotary = _norm_args(q, k, q_w, k_w, positions, inv_freq)
    ld = [_token_stride(t) if T else 0 for t in (q, k)]
    oq = _out(out_q, q.shape, q.dtype, q.device)
    ok = _out(out_k, k.shape, k.dtype, k.device)
    with _on(q.device):
        st = lib().gdn_qk_norm_rope(_ptr(q), _ptr(k), _dtype_code(q), T, H, k.shape[1], D, ld[0], ld[1], _ptr(q_w),
                                    _ptr(k_w), float(eps), _ptr(positions), _ptr(inv_freq), rotary,
                                    int(interleaved), _ptr(oq), _ptr(ok), _stream(q.device))
    _check(st, "gdn_qk_norm_rope")
    return oq, ok


def qk_norm_rope_cache(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_w: torch.Tensor, k_w: torch.Tensor,
                       positions: torch.Tensor, inv_freq: torch.Tensor, cache: KVCache, page_table: torch.Tensor,
                       seq_lens: torch.Tensor, cu_seqlens: torch.Tensor, *, eps: float = 1e-6,
                       interleaved: bool = False, out_q: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qk_norm_rope with the keys and the values v [T, Hk, D] written to the
    cache in the same pass, at the last positions of their sequences
    (seq_lens counts them). Returns q."""
    T, H, D, rotary = _norm_args(q, k, q_w, k_w, positions, inv_freq)
    if v.shape != k.shape or v.dtype != q.dtype or tuple(k.shape[1:]) != (cache.k.shape[1], cache.k.shape[3]):
        raise ValueError("k and v must be [T, Hk, D] of one dtype, Hk and D the cache's")
    _same_device(q.device, v, cache.k, page_table, seq_lens, cu_seqlens)
    ld = [_token_stride(t) if T else 0 for t in (q, k, v)]
    oq = _out(out_q, q.shape, q.dtype, q.device)
    c = _cache_arg(cache)
    with _on(q.device):
        st = lib().gdn_qk_norm_rope_cache(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), T, H, ld[0], ld[1], ld[2],
                                          _ptr(q_w), _ptr(k_w), float(eps), _ptr(positions), _ptr(inv_freq), rotary,
                                          int(interleaved), ctypes.byref(c), *_pages(page_table, seq_lens, cu_seqlens),
                                          _ptr(oq), _stream(q.device))
    _check(st, "gdn_qk_norm_rope_cache")
    return oq


def kv_cache_write(k: torch.Tensor, v: torch.Tensor, cache: KVCache, page_table: torch.Tensor,
                   seq_lens: torch.Tensor, cu_seqlens: torch.Tensor) -> None:
    """Writes k, v [T, Hk, D] (bf16 or fp32, token-strided views allowed) at the
    last positions of their sequences, quantised where the cache is."""
    T = k.shape[0]
    if k.dim() != 3 or v.shape != k.shape or v.dtype != k.dtype \
            or tuple(k.shape[1:]) != (cache.k.shape[1], cache.k.shape[3]):
        raise ValueError("k and v must be [T, Hk, D] of one dtype, Hk and D the cache's")
    _same_device(k.device, v, cache.k, page_table, seq_lens, cu_seqlens)
    ld = [_token_stride(t) if T else 0 for t in (k, v)]
    c = _cache_arg(cache)
    with _on(k.device):
        st = lib().gdn_kv_write(_ptr(k), _ptr(v), _dtype_code(k), T, ld[0], ld[1], ctypes.byref(c),
                                *_pages(page_table, seq_lens, cu_seqlens), _stream(k.device))
    _check(st, "gdn_kv_write")


def kv_cache_read(cache: KVCache, page_table: torch.Tensor, seq_lens: torch.Tensor, cu_seqlens: torch.Tensor, *,
                  n_tokens: int, dtype: torch.dtype = torch.bfloat16, out_k: Optional[torch.Tensor] = None,
                  out_v: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Keys and values of each sequence's last cu_seqlens[n+1] - cu_seqlens[n]
    positions (cu_seqlens the running sum of seq_lens: all of them) as dense
    k, v [n_tokens, Hk, D] of dtype bf16 or fp32. Rows behind cu_seqlens[N] are
    left as they are."""
    c = _cache_arg(cache)
    dev = cache.k.device
    _same_device(dev, page_table, seq_lens, cu_seqlens)
    shape = (int(n_tokens), cache.k.shape[1], cache.k.shape[3])
    k, v = _out(out_k, shape, dtype, dev), _out(out_v, shape, dtype, dev)
    with _on(dev):
        st = lib().gdn_kv_read(ctypes.byref(c), *_pages(page_table, seq_lens, cu_seqlens), shape[0], _dtype_code(k),
                               _ptr(k), _ptr(v), _stream(dev))
    _check(st, "gdn_kv_read")
    return k, v


def kv_cache_accept(cache: KVCache, page_table: torch.Tensor, seq_lens: torch.Tensor, cu_seqlens: torch.Tensor,
                    accepted: torch.Tensor, *, out_seq_lens: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Keeps the accepted path of every draft: accepted [N, M] int32 holds each
    sequence's accepted nodes, increasing, then -1s. Their cache rows move to the
    front of the draft, in place. Returns the new seq_lens."""
    c = _cache_arg(cache)
    dev = cache.k.device
    pages = _pages(page_table, seq_lens, cu_seqlens)
    if accepted.dim() != 2 or accepted.shape[0] != pages[-1] or accepted.dtype != torch.int32:
        raise ValueError("accepted must be [N, M] int32")
    _cuda(accepted)
    _same_device(dev, page_table, seq_lens, cu_seqlens, accepted)
    out = _out(out_seq_lens, seq_lens.shape, torch.int32, dev)
    with _on(dev):
        st = lib().gdn_kv_accept(ctypes.byref(c), *pages, _ptr(accepted), accepted.shape[1], _ptr(out), _stream(dev))
    _check(st, "gdn_kv_accept")
    return out


def tree_attention_workspace_size(cache: KVCache, N: int, H: int, max_nodes: int) -> int:
    """Bytes of workspace for tree_attention on the current device."""
    return int(lib().gdn_tree_attention_workspace_size(ctypes.byref(_cache_arg(cache)), N, H, max_nodes))


def tree_attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, seq_lens: torch.Tensor,
                   cu_seqlens: torch.Tensor, *, max_nodes: int, mask: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, gate: Optional[torch.Tensor] = None, return_lse: bool = False,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Attention of the drafted tokens q [T, H, D] bf16 (a token-strided view is
    fine) over their sequences' cached positions, the drafted ones included:
    each node sees all of the context before the draft, and the drafted nodes
    whose bit its mask [T] int64 has (see tree_mask; None: a chain, which for
    one token is a plain decode step). max_nodes (1 to 64) bounds the drafted
    tokens of a sequence. scale defaults to D^-1/2; gate [T, H, D] bf16
    multiplies the output by its sigmoid. Returns o, or (o, lse [T, H] fp32).
    Calls that may overlap on the GPU need a workspace each (by default every
    call allocates its own)."""
    c = _cache_arg(cache)
    dev = q.device
    if q.dim() != 3 or q.shape[2] != cache.k.shape[3]:
        raise ValueError("q must be [T, H, D], D the cache's")
    T, H, D = q.shape
    if mask is not None and (tuple(mask.shape) != (T,) or mask.dtype != torch.int64):
        raise ValueError("mask must be [T] int64")
    if gate is not None and (gate.shape != q.shape or gate.dtype != q.dtype):
        raise ValueError("gate must be [T, H, D] in the dtype of q")
    pages = _pages(page_table, seq_lens, cu_seqlens)
    ld = _token_stride(q) if T else 0
    _cuda(mask, gate, workspace)
    _same_device(dev, cache.k, page_table, seq_lens, cu_seqlens, mask, gate, workspace)
    o = _out(out, q.shape, q.dtype, dev)
    lse = torch.empty((T, H), dtype=torch.float32, device=dev) if return_lse else None
    with _on(dev):
        if workspace is None:
            size = lib().gdn_tree_attention_workspace_size(ctypes.byref(c), pages[-1], H, max_nodes)
            workspace = torch.empty(int(size), dtype=torch.uint8, device=dev)
        st = lib().gdn_tree_attention(_ptr(q), _dtype_code(q), T, ld, H, ctypes.byref(c), *pages, _ptr(mask),
                                      int(max_nodes), float(D ** -0.5 if scale is None else scale), _ptr(gate),
                                      _ptr(o), _ptr(lse), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(dev))
    _check(st, "gdn_tree_attention")
    return (o, lse) if return_lse else o
