"""The softmax-attention layers between the linear ones, for serving: q/k norm
with the rotation, the paged key/value cache and the attention of drafted
tokens over it. The tensors' checks and the calls of the C ABI (include/gdn.h)
stand in C++ (csrc/binding.cpp): on the host a call then costs about as much as
its launch.

A decode step of such a layer:

    q = qk_norm_rope_cache(q, k, v, q_w, k_w, positions, inv_freq, cache, page_table, seq_lens, cu_seqlens)
    o = tree_attention(q, cache, page_table, seq_lens, cu_seqlens, mask=mask, max_nodes=nodes, gate=gate)
    seq_lens = kv_cache_accept(cache, page_table, seq_lens, cu_seqlens, accepted)   # after verification
"""
from __future__ import annotations

import ctypes
import importlib
import os
from typing import NamedTuple, Optional, Tuple

import torch

from . import _HERE, GDNError, lib

_ENTRIES = ("gdn_qk_norm_rope", "gdn_qk_norm_rope_cache", "gdn_kv_write", "gdn_kv_read", "gdn_kv_accept",
            "gdn_tree_attention_workspace_size", "gdn_tree_attention")
_bound = None


def _binding():
    """The C++ entry points, bound to the loaded libgdn.so."""
    global _bound
    if _bound is None:
        if not os.path.exists(os.path.join(_HERE, "_binding.so")):
            raise RuntimeError("_binding.so is missing: build it with `python -m gated_deltanet_linear_silu_b200.build`")
        from . import build

        if not build.binding_matches():  # (before it is loaded)
            raise RuntimeError(f"_binding.so is not the {build.binding_tag()}: "
                               "build it with `python -m gated_deltanet_linear_silu_b200.build`")
        library = lib()  # refuses another ABI version
        module = importlib.import_module("._binding", __package__)
        module.bind(*(ctypes.cast(getattr(library, name), ctypes.c_void_p).value for name in _ENTRIES), GDNError)
        _bound = module
    return _bound


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
    return (_bound or _binding()).qk_norm_rope(q, k, q_w, k_w, positions, inv_freq, eps, interleaved, out_q, out_k)


def qk_norm_rope_cache(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_w: torch.Tensor, k_w: torch.Tensor,
                       positions: torch.Tensor, inv_freq: torch.Tensor, cache: KVCache, page_table: torch.Tensor,
                       seq_lens: torch.Tensor, cu_seqlens: torch.Tensor, *, eps: float = 1e-6,
                       interleaved: bool = False, out_q: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qk_norm_rope with the keys and the values v [T, Hk, D] written to the
    cache in the same pass, at the last positions of their sequences
    (seq_lens counts them). Returns q."""
    return (_bound or _binding()).qk_norm_rope_cache(q, k, v, q_w, k_w, positions, inv_freq, *cache, page_table,
                                                     seq_lens, cu_seqlens, eps, interleaved, out_q)


def kv_cache_write(k: torch.Tensor, v: torch.Tensor, cache: KVCache, page_table: torch.Tensor,
                   seq_lens: torch.Tensor, cu_seqlens: torch.Tensor) -> None:
    """Writes k, v [T, Hk, D] (bf16 or fp32, token-strided views allowed) at the
    last positions of their sequences, quantised where the cache is."""
    (_bound or _binding()).kv_write(k, v, *cache, page_table, seq_lens, cu_seqlens)


def kv_cache_read(cache: KVCache, page_table: torch.Tensor, seq_lens: torch.Tensor, cu_seqlens: torch.Tensor, *,
                  n_tokens: int, dtype: torch.dtype = torch.bfloat16, out_k: Optional[torch.Tensor] = None,
                  out_v: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Keys and values of each sequence's last cu_seqlens[n+1] - cu_seqlens[n]
    positions (cu_seqlens the running sum of seq_lens: all of them) as dense
    k, v [n_tokens, Hk, D] of dtype bf16 or fp32. Rows behind cu_seqlens[N] are
    left as they are."""
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError(f"unsupported dtype {dtype} (bf16 or fp32)")
    return (_bound or _binding()).kv_read(*cache, page_table, seq_lens, cu_seqlens, n_tokens, dtype is torch.bfloat16,
                                          out_k, out_v)


def kv_cache_accept(cache: KVCache, page_table: torch.Tensor, seq_lens: torch.Tensor, cu_seqlens: torch.Tensor,
                    accepted: torch.Tensor, *, out_seq_lens: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Keeps the accepted path of every draft: accepted [N, M] int32 holds each
    sequence's accepted nodes, increasing, then -1s. Their cache rows move to the
    front of the draft, in place. Returns the new seq_lens."""
    return (_bound or _binding()).kv_accept(*cache, page_table, seq_lens, cu_seqlens, accepted, out_seq_lens)


def tree_attention_workspace_size(cache: KVCache, N: int, H: int, max_nodes: int) -> int:
    """Bytes of workspace for tree_attention over this cache on the current device."""
    P, Hk, page, D = cache.k.shape
    return _workspace_size(P, page, Hk, D, cache.k.dtype == torch.float8_e4m3fn, N, H, max_nodes)


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page", ctypes.c_int),
                ("Hk", ctypes.c_int), ("D", ctypes.c_int), ("dtype", ctypes.c_int)]


def _workspace_size(n_pages, page, Hk, D, e4m3, N, H, max_nodes) -> int:
    c = _CacheStruct(None, None, None, None, n_pages, page, Hk, D, 2 if e4m3 else 1)
    return int(lib().gdn_tree_attention_workspace_size(ctypes.byref(c), N, H, max_nodes))


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
    return (_bound or _binding()).tree_attention(q, *cache, page_table, seq_lens, cu_seqlens, max_nodes, mask, scale,
                                                 gate, return_lse, out, workspace)
