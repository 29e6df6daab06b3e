"""fp64 restatement of the softmax-attention layer's operators, for the tests:
the q/k norm with the rotation, e4m3 rounding, and attention of a drafted tree
over given keys and values. Plain torch on the CPU, sequence by sequence; no
code of the package."""
from __future__ import annotations

import math

import torch


def norm(x: torch.Tensor, w: torch.Tensor, eps: float) -> torch.Tensor:
    """RMSNorm over the last axis, times w."""
    x = x.double()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()


def rotate(y: torch.Tensor, pos: torch.Tensor, inv_freq: torch.Tensor, interleaved: bool) -> torch.Tensor:
    """Rotation of the first 2 len(inv_freq) elements of y [T, H, D]."""
    out = y.clone()
    half = inv_freq.numel()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = (pos.double() * inv_freq[i].double())[:, None]
        out[..., a] = y[..., a] * torch.cos(t) - y[..., b] * torch.sin(t)
        out[..., b] = y[..., b] * torch.cos(t) + y[..., a] * torch.sin(t)
    return out


def pair_size(y: torch.Tensor, half: int, interleaved: bool) -> torch.Tensor:
    """|a| + |b| of the pair that each element belongs to (|y| where unrotated)."""
    s = y.abs().clone()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        s[..., a] = s[..., b] = y[..., a].abs() + y[..., b].abs()
    return s


def attention(q, k, v, base: int, masks, scale: float, gate=None):
    """One sequence. q [n, H, D], k, v [L, Hk, D], node i sees positions below
    base and base + j for the set bits j of masks[i]. Returns (o, lse, and two
    sizes that bound the rounding: sum_j p_j |v_j| and max_j scale |q|.|k_j|)."""
    n, H, D = q.shape
    L, Hk, _ = k.shape
    o, lse = torch.zeros(n, H, D, dtype=torch.float64), torch.full((n, H), -math.inf, dtype=torch.float64)
    mass, size = torch.zeros_like(o), torch.zeros_like(lse)
    for i in range(n):
        seen = list(range(base)) + [base + j for j in range(L - base) if int(masks[i]) >> j & 1]
        if not seen:
            continue
        for h in range(H):
            kk, vv = k[seen, h * Hk // H].double(), v[seen, h * Hk // H].double()
            s = kk @ q[i, h].double() * scale
            z = torch.logsumexp(s, 0)
            p = torch.exp(s - z)
            lse[i, h] = z
            o[i, h] = (p[:, None] * vv).sum(0)
            mass[i, h] = (p[:, None] * vv.abs()).sum(0)
            size[i, h] = (kk.abs() @ q[i, h].double().abs() * scale).max()
    if gate is not None:
        g = 1 / (1 + torch.exp(-gate.double()))
        o, mass = o * g, mass * g
    return o, lse, mass, size
