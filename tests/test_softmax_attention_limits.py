"""The softmax-attention layer's calls where they are easiest to get wrong:
drafts that end inside a CTA's stretch of work, inputs that are not finite on
either attention kernel, buffers that overlap. Tolerances and helpers are those
of test_softmax_attention.py."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_linear_silu_b200 as gdn
from oracle import attention as ref
from test_softmax_attention import (BF, DEV, E, F8, F32, Pool, _cuda, _status, check_attention, close,  # noqa: F401
                                    half_step, rnd, status_bad, trees)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- drafts that end inside a stretch

def elapsed_ms(call):
    call()
    torch.cuda.synchronize()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    call()
    b.record()
    b.synchronize()
    return a.elapsed_time(b)


@pytest.mark.parametrize("held", [BF, F8])
@pytest.mark.parametrize("lens,nodes,H,Hk,D", [
    ([2048] * 16, [16] * 16, 32, 8, 128), ([1024] * 32, [24] * 32, 32, 8, 128), ([516] * 64, [16] * 64, 32, 8, 128),
    ([216] * 128, [16] * 128, 32, 8, 128), ([194] * 256, [64] * 256, 32, 8, 128),
    ([2000] * 24, [17] * 24, 8, 2, 256), ([1017] * 24, [17] * 24, 8, 2, 256), ([700] * 40, [9] * 40, 16, 4, 64),
    ([200 + 137 * i % 3000 for i in range(40)], [1 + i % 33 for i in range(40)], 16, 4, 64),
    ([70 + 137 * i % 1500 for i in range(48)], [min(64, 1 + 7 * i % 64) for i in range(48)], 16, 4, 128),
    ([200 + 137 * i % 3000 for i in range(40)], [1 + i % 33 for i in range(40)], 8, 2, 256),
])
def test_tree_attention_ends_inside_a_stretch(lens, nodes, H, Hk, D, held):
    """More than sixteen query rows, sequences that end a few tiles before a CTA's
    work does: the results, and no wait that runs out (at the least a second; a
    call's work here is under two milliseconds)."""
    pool = Pool(lens, nodes, Hk, D, 64, held, fill=141)
    q = rnd(142, sum(nodes), H, D, dtype=BF).to(DEV)
    mask = trees(nodes, 12)
    call = lambda: gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=max(nodes), mask=mask.to(DEV), return_lse=True)
    assert elapsed_ms(call) < 200
    o, lse = call()
    gdn.check_device_status(DEV)
    small = sorted(range(len(lens)), key=lambda n: lens[n] * nodes[n])
    check_attention(pool, q, o, lse, mask, D ** -0.5, rows=[small[0], small[len(small) // 3]])


# ---------------------------------------------------------------- inputs that are not finite

@pytest.mark.parametrize("heads,D,lens,c", [(2, 128, 44, 8), (1, 64, 3007, 5), (4, 256, 45, 3), (2, 256, 641, 2),
                                            (4, 128, 44, 8), (8, 64, 3007, 5), (16, 256, 641, 2), (8, 256, 45, 3)])
def test_tree_attention_non_finite_context(heads, D, lens, c):
    """Context values that are not finite reach every row, also where their tokens
    stand right before the draft (which is held back there); up to sixteen query
    rows and more."""
    pool = Pool([lens], [c], 1, D, 16, BF, fill=151)
    base = lens - c
    for at, element, value in ((base - 1, 3, math.inf), (base - 2, 5, math.nan), (base // 2, 9, -math.inf)):
        page, row = (int(x) for x in pool.spots(0, at))
        pool.cache.v[page, 0, row, element] = value
    q = rnd(152, c, heads, D, dtype=BF).to(DEV)
    mask = trees([c], 13)
    o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=c, mask=mask.to(DEV), return_lse=True)
    assert (o[..., 3] == math.inf).all() and o[..., 5].isnan().all() and (o[..., 9] == -math.inf).all()
    rest = [e for e in range(D) if e not in (3, 5, 9)]
    assert o[..., rest].isfinite().all() and lse.isfinite().all()
    k, v = (pool.rows(0, range(lens), name) for name in ("k", "v"))
    want, z, mass, size = ref.attention(q.cpu(), k, v.nan_to_num(0, 0, 0), base, mask, D ** -0.5)
    s, u = ((D + 8) * E * size + 8 * E)[..., None], half_step(BF)
    close(o[..., rest], want[..., rest], ((u + 2 * s + 2.0 ** -9) * mass * (1 + u) + u * want.abs())[..., rest])
    close(lse, z, s[..., 0] + 2.0 ** -9 + 8 * E * z.abs())
