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
