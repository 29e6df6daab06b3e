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


@pytest.mark.parametrize("held", [F8, BF])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("length", [40, 72, 128, 5000])
def test_many_rows_non_finite_behind_the_mask(held, D, length):
    """test_tree_attention_non_finite_behind_the_mask with 32 query rows: NaN and
    infinities in a node that a row does not see do not reach it; in one that it
    sees, they do. Rows behind the sequence hold NaN as well."""
    c = 8
    pool = Pool([length], [c], 1, D, 16, held, fill=161)
    base = length - c

    def put(name, node, value, element=None):
        page, row = (int(x) for x in pool.spots(0, base + node))
        if held == F8:
            getattr(pool.cache, name + "_scale")[page, :, row] = value
        else:
            getattr(pool.cache, name)[page, :, row, slice(None) if element is None else element] = value

    mask = torch.tensor([0b1, 0b11, 0b101, 0b1001, 0b10001, 0b110001, 0b1010001, 0b10111001], dtype=torch.int64)
    q = rnd(162, c, 4, D, dtype=BF).to(DEV)
    clean, clean_lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=c, mask=mask.to(DEV), return_lse=True)
    check_attention(pool, q, clean, clean_lse, mask, D ** -0.5)
    put("v", 1, math.nan)
    put("k", 2, math.nan)
    if held == BF:
        put("v", 3, math.inf, 33)
    else:
        put("k", 1, math.inf)  # a scale that no write leaves, in the node whose values are NaN
    if length % 16:
        page = pool.ids[0, length // 16]
        for name in ("k", "v"):
            if held == F8:
                getattr(pool.cache, name + "_scale")[page, :, length % 16:] = math.nan
                getattr(pool.cache, name).view(torch.uint8)[page, :, length % 16:] = 0x7F
            else:
                getattr(pool.cache, name)[page, :, length % 16:] = math.nan
    o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=c, mask=mask.to(DEV), return_lse=True)
    assert o[1].isnan().all() and o[2].isnan().all() and lse[2].isnan().all()
    same = [0, 3, 4, 5, 6, 7] if held == F8 else [0, 4, 5, 6]
    assert torch.equal(o[same], clean[same]) and torch.equal(lse[same], clean_lse[same])
    if held == BF:
        assert lse[1].isfinite().all()
        for t in (3, 7):
            assert (o[t, :, 33] == math.inf).all() and torch.equal(lse[t], clean_lse[t])
            rest = [e for e in range(D) if e != 33]
            assert torch.equal(o[t][:, rest], clean[t][:, rest])


@pytest.mark.parametrize("held", [F8, BF])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows_extreme_scores(held, D):
    """test_tree_attention_extreme_scores with 32 query rows. A row's numerators
    are off by at most 2 s, s its scores' error; where that passes one they may be
    anything between none and all, but stay weights: the output is bounded by the
    largest value."""
    pool = Pool([300, 70], [4, 4], 1, D, 16, held, fill=163)
    q = rnd(164, 8, 8, D, dtype=BF, scale=300.0).to(DEV)
    mask = trees([4, 4], 14)
    o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=4, mask=mask.to(DEV), scale=30.0, return_lse=True)
    for n, (l, rows) in enumerate(((300, slice(0, 4)), (70, slice(4, 8)))):
        k, v = pool.rows(n, range(l), "k"), pool.rows(n, range(l), "v")
        want, z, mass, size = ref.attention(q[rows].cpu(), k, v, l - 4, mask[rows], 30.0)
        assert (o[rows].cpu().double().abs() <= v.abs().amax() * (1 + 2.0 ** -6)).all()
        assert ((lse[rows].cpu().double() - z).abs() <= (D + 16) * E * size + 8 * E * z.abs() + 2.0 ** -9).all()
    if held == BF:  # every key at minus infinity
        pool.cache.k[:] = 0
        pool.cache.k[..., 0] = -math.inf
        q = torch.zeros(8, 8, D, dtype=BF, device=DEV)
        q[..., 0] = 1
        o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=4, mask=mask.to(DEV), return_lse=True)
        assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("held", [F8, BF])
@pytest.mark.parametrize("D", [128, 256])
def test_many_rows_growing_scores(held, D):
    """Scores that rise and fall by hundreds along the context: the running
    reference moves many times, on either parity of the tiles."""
    L, c = 2100, 6
    pool = Pool([L], [c], 1, D, 32, held)
    k, v = (rnd(165 + i, L, 1, D) for i in (0, 1))
    wave = torch.cumsum(torch.where(torch.rand(L, generator=torch.Generator().manual_seed(3)) < 0.5, -1.0, 1.0), 0)
    k[:, 0, 0] = wave * 8 + torch.arange(L) / 16
    whole = (pool.table, pool.lens, torch.tensor([0, L], dtype=torch.int32, device=DEV))
    gdn.kv_cache_write(k.to(DEV), v.to(DEV), pool.cache, *whole)
    q = rnd(167, c, 4, D, dtype=BF)
    q[..., 0] = 16
    q = q.to(DEV)
    mask = trees([c], 15)
    o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=c, mask=mask.to(DEV), return_lse=True)
    check_attention(pool, q, o, lse, mask, D ** -0.5)


@pytest.mark.parametrize("held", [F8, BF])
@pytest.mark.parametrize("page", [16, 64])
def test_many_rows_bad_sequences(held, page):
    """test_tree_attention_bad_sequences with 32 query rows and more: what the
    loader and the converters do about a page that does not exist, in the context
    and in the draft."""
    for what in ("nodes", "short", "page", "last"):
        pool = Pool([150, 260], [8, 9], 1, 64, page, held, fill=171)
        q = rnd(172, 17, 8, 64, dtype=BF).to(DEV)
        if what == "short":
            pool.lens[0] = 100000
        if what == "page":
            pool.table[0, 1] = 1 << 30
        if what == "last":
            pool.table[0, 149 // page] = -1
        if what == "nodes":
            pool.cu[1], pool.cu[2] = 8, 8 + 40
            q = rnd(172, 48, 8, 64, dtype=BF).to(DEV)
            pool.host_lens, pool.counts = [150, 260], [8, 40]
        out = torch.full(q.shape, 7.0, dtype=BF, device=DEV)
        o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=9, out=out, return_lse=True)
        status_bad()
        if what == "nodes":
            assert (o[8:] == 7).all()
        elif what == "short":
            assert (o[:8] == 7).all()
        check_attention(pool, q, o, lse, None, 0.125, rows=[0 if what == "nodes" else 1])


@pytest.mark.parametrize("held", [F8, BF])
@pytest.mark.parametrize("nodes,H", [(2, 8), (5, 32)])
def test_many_pages_past_32_bits(held, nodes, H):
    """Rows whose byte and element offsets pass 2^32, both kernels and cache types."""
    P, page, Hk, D = 18000, 128, 8, 256
    shape = (P, Hk, page, D)
    cache = gdn.KVCache(*(torch.empty(shape, dtype=held, device=DEV) for _ in range(2)),
                        *((torch.empty(shape[:3], dtype=F32, device=DEV) for _ in range(2)) if held == F8 else ()))
    table = torch.tensor([[P - 1, 3, P - 2]], dtype=torch.int32, device=DEV)
    lens, cu = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([300], [0, 300]))
    k, v = (rnd(s, 300, Hk, D, dtype=BF) for s in (181, 182))
    gdn.kv_cache_write(k.to(DEV), v.to(DEV), cache, table, lens, cu)
    a, b = gdn.kv_cache_read(cache, table, lens, cu, n_tokens=300, dtype=F32)
    q = rnd(183, nodes, H, D, dtype=BF).to(DEV)
    draft = torch.tensor([0, nodes], dtype=torch.int32, device=DEV)
    o = gdn.tree_attention(q, cache, table, lens, draft, max_nodes=nodes)
    want, z, mass, size = ref.attention(q.cpu(), a.cpu(), b.cpu(), 300 - nodes, [(2 << i) - 1 for i in range(nodes)], D ** -0.5)
    s = ((D + 8) * E * size + 8 * E)[..., None]
    u = half_step(BF)
    close(o, want, (u + 2 * s + 2.0 ** -9) * mass * (1 + u) + u * want.abs())


# ---------------------------------------------------------------- buffers that overlap

def test_overlapping_tensors_are_refused():
    """Outputs that lie on what is read, or on one another; in place and side by
    side in one buffer they are fine."""
    T, H, D = 6, 2, 64
    w, pos, f = torch.ones(D, device=DEV), torch.arange(T, dtype=torch.int32, device=DEV), gdn.rope_inv_freq(32, device=DEV)
    room = rnd(191, 6 * T, H, D, dtype=BF).to(DEV)
    q, k, v, a, b = (room[i * T:(i + 1) * T] for i in range(5))
    for kw in (dict(out_q=k), dict(out_k=q), dict(out_q=a, out_k=a), dict(out_q=room[1:T + 1]), dict(out_q=a, out_k=room[3 * T + 1:4 * T + 1])):
        with pytest.raises(gdn.GDNError):
            gdn.qk_norm_rope(q, k, w, w, pos, f, **kw)
    want = gdn.qk_norm_rope(q, k, w, w, pos, f)
    got = gdn.qk_norm_rope(q, k, w, w, pos, f, out_q=a, out_k=b)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    pool = Pool([20], [T], H, D, 16, BF, fill=192)
    cache, pages = pool.cache, pool.where
    for kw in (dict(out_q=k), dict(out_q=v), dict(out_q=room[1:T + 1]), dict(out_q=cache.k.view(-1)[:T * H * D].view(T, H, D))):
        with pytest.raises(gdn.GDNError):
            gdn.qk_norm_rope_cache(q, k, v, w, w, pos, f, cache, *pages, **kw)
    with pytest.raises(gdn.GDNError):
        gdn.kv_cache_write(cache.k.view(-1)[:T * H * D].view(T, H, D), v, cache, *pages)
    with pytest.raises(gdn.GDNError):
        gdn.kv_cache_write(k, v, cache._replace(v=cache.k), *pages)
    with pytest.raises(gdn.GDNError):
        gdn.kv_cache_read(cache, *pages, n_tokens=T, out_k=a, out_v=room[3 * T + 1:4 * T + 1])
    lens = torch.tensor([20, 0], dtype=torch.int32, device=DEV)
    with pytest.raises(gdn.GDNError):
        gdn.kv_cache_accept(cache, pages[0], lens[:1], pages[2], torch.zeros((1, 1), dtype=torch.int32, device=DEV),
                            out_seq_lens=pages[2][1:])
    got = gdn.kv_cache_accept(cache, pages[0], lens[:1], pages[2], torch.zeros((1, 1), dtype=torch.int32, device=DEV),
                              out_seq_lens=lens[1:])
    assert lens.tolist() == [20, 15] and got.data_ptr() == lens[1:].data_ptr()
    for kw in (dict(out=q), dict(out=room[1:T + 1]), dict(gate=v, out=v), dict(out=a, workspace=room.view(torch.uint8))):
        with pytest.raises(gdn.GDNError):
            gdn.tree_attention(q, cache, *pages, max_nodes=T, **kw)
    want = gdn.tree_attention(q, cache, *pages, max_nodes=T)
    assert torch.equal(gdn.tree_attention(q, cache, *pages, max_nodes=T, out=a), want)


# ---------------------------------------------------------------- lengths

@pytest.mark.parametrize("held", [F8, BF])
@pytest.mark.parametrize("heads", [4, 32])  # either kernel
def test_tree_attention_refuses_lengths_next_to_32_bits(held, heads):
    """A length whose last tile would end past 2^31 is skipped and reported; the
    other sequence is done."""
    pool = Pool([40, 70], [1, 1], 1, 64, 1024, held, fill=201)
    wide = torch.zeros((2, 1 << 21), dtype=torch.int32, device=DEV)  # 2^31 positions of pages that exist
    wide[1, 0] = int(pool.ids[1, 0])
    q = rnd(202, 2, heads, 64, dtype=BF).to(DEV)
    for length in (2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 1023):
        pool.lens[0] = length
        out = torch.full(q.shape, 7.0, dtype=BF, device=DEV)
        o, lse = gdn.tree_attention(q, pool.cache, wide, pool.lens, pool.cu, max_nodes=1, out=out, return_lse=True)
        status_bad()
        assert (o[0] == 7).all()
        check_attention(pool, q, o, lse, None, 0.125, rows=[1])


# ---------------------------------------------------------------- f16 operands of an e4m3 cache

@pytest.mark.parametrize("held", [F8, BF])
@pytest.mark.parametrize("heads", [4, 32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("log2_outlier", [12, 17, 20, 24])
def test_tree_attention_beside_an_outlier_in_the_queries(heads, D, log2_outlier, held):
    """A query element far above the others, at a channel where the keys are zero:
    the scores are the other elements', to all their bits."""
    L = 300
    pool = Pool([L], [1], 1, D, 16, held)
    k, v = rnd(221, L, 1, D), rnd(222, L, 1, D)
    k[..., 5] = 0
    whole = (pool.table, pool.lens, torch.tensor([0, L], dtype=torch.int32, device=DEV))
    gdn.kv_cache_write(k.to(DEV), v.to(DEV), pool.cache, *whole)
    q = rnd(223, 1, heads, D, dtype=BF)
    q[..., 5] = 2.0 ** log2_outlier
    q = q.to(DEV)
    o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=1, return_lse=True)
    k, v = (pool.rows(0, range(L), name) for name in ("k", "v"))
    want, z, mass, size = ref.attention(q.cpu(), k, v, L - 1, [1], D ** -0.5)
    s, u = ((D + 8) * E * size + 8 * E)[..., None], half_step(BF)
    close(o, want, (u + 2 * s + 2.0 ** -9) * mass * (1 + u) + u * want.abs())
    close(lse, z, s[..., 0] + 16 * E * (1 + z.abs()))  # (300 additions of a row: under a dozen to a chain)
@pytest.mark.parametrize("heads", [4, 32])  # either kernel
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("log2_ratio", [-14.3, -17.2, -20.6])
def test_tree_attention_beside_a_dominating_token(heads, D, log2_ratio):
    """One context token takes nearly all of a row's weight but holds a value in one
    element only: the others' sums, all of small numerators that round alike, keep
    their bits. (The numerators are at least 2^-21 of the largest: eleven bits in f16
    where that is at least 2^7, ten where they reach below the normal range; the
    tolerance counts eight.)"""
    L, N = 192, 1200  # as many sequences, all on the same pages, as leave most of them whole to a CTA
    pool = Pool([L], [1], 1, D, 32, F8)
    k, v = torch.zeros(L, 1, D), rnd(211, 1, 1, D).repeat(L, 1, 1)
    k[20, 0, 0] = -log2_ratio * math.log(2) / D ** -0.5
    v[20] = 0
    v[20, 0, 0] = float(v[0].abs().max())
    whole = (pool.table, pool.lens, torch.tensor([0, L], dtype=torch.int32, device=DEV))
    gdn.kv_cache_write(k.to(DEV), v.to(DEV), pool.cache, *whole)
    q = torch.zeros(N, heads, D, dtype=BF, device=DEV)
    q[..., 0] = 1
    o, lse = gdn.tree_attention(q, pool.cache, pool.table.repeat(N, 1), pool.lens.repeat(N),
                                torch.arange(N + 1, dtype=torch.int32, device=DEV), max_nodes=1, return_lse=True)
    k, v = (pool.rows(0, range(L), name) for name in ("k", "v"))
    want, z, mass, size = ref.attention(q[:1].cpu(), k, v, L - 1, [1], D ** -0.5)
    s, u = ((D + 8) * E * size + 8 * E)[..., None], half_step(BF)
    close(o, want.expand(N, -1, -1), ((u + 2 * s + 2.0 ** -9) * mass * (1 + u) + u * want.abs()).expand(N, -1, -1))
    close(lse, z.expand(N, -1), (s[..., 0] + 16 * E * (1 + z.abs())).expand(N, -1))




@pytest.mark.parametrize("heads", [4, 32])
def test_tree_attention_over_values_of_all_sizes(heads):
    """Rows of values that are zero, of ordinary size, tiny and huge: the reference
    follows their scales, the weights without them stay finite."""
    L, D = 3000, 128
    for sizes in ((0.0,), (0.0, 1.0), (1e-30, 1e30), (1e-38, 1.0, 0.0), (3e38, 1e-3)):
        pool = Pool([L], [1], 1, D, 32, F8)
        k, v = rnd(231, L, 1, D), rnd(232, L, 1, D).clamp(-1, 1)
        v *= torch.tensor([sizes[i * 7919 % len(sizes)] for i in range(L)])[:, None, None]
        whole = (pool.table, pool.lens, torch.tensor([0, L], dtype=torch.int32, device=DEV))
        gdn.kv_cache_write(k.to(DEV), v.to(DEV), pool.cache, *whole)
        q = rnd(233, 1, heads, D, dtype=BF).to(DEV)
        o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=1, return_lse=True)
        check_attention(pool, q, o, lse, None, D ** -0.5)


# ---------------------------------------------------------------- odd Python arguments

def test_flags_without_a_truth_value():
    """What has no truth value raises its own error, and no result comes with it."""
    T, H, D = 2, 2, 64
    q, w = rnd(241, T, H, D, dtype=BF).to(DEV), torch.ones(D, device=DEV)
    pos, f = torch.arange(T, dtype=torch.int32, device=DEV), gdn.rope_inv_freq(32, device=DEV)
    pool = Pool([20], [T], H, D, 16, BF, fill=242)
    both = torch.ones(2)
    with pytest.raises(RuntimeError, match="ambiguous"):
        gdn.qk_norm_rope(q, q.clone(), w, w, pos, f, interleaved=both)
    with pytest.raises(RuntimeError, match="ambiguous"):
        gdn.qk_norm_rope_cache(q, q.clone(), q.clone(), w, w, pos, f, pool.cache, *pool.where, interleaved=both)
    with pytest.raises(RuntimeError, match="ambiguous"):
        gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=T, return_lse=both)


def test_head_counts_past_32_bits_are_refused():
    """Counted in 32 bits by the C ABI: 2^32 + 2 heads must not pass as two. (No
    tokens, so that there is nothing to allocate.)"""
    w, pos, f = torch.ones(64, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV), gdn.rope_inv_freq(32, device=DEV)
    many, two = (torch.empty((0, h, 64), dtype=BF, device=DEV) for h in ((1 << 32) + 2, 2))
    assert gdn.qk_norm_rope(two, two, w, w, pos, f)[0].shape == (0, 2, 64)
    for q, k in ((many, two), (two, many)):
        with pytest.raises(ValueError):
            gdn.qk_norm_rope(q, k, w, w, pos, f)


# ---------------------------------------------------------------- fewer rows than the bounds count

@pytest.mark.parametrize("held", [F8, BF])
def test_fewer_packed_rows_than_tokens_are_reported(held):
    """Keys and values that end before cu_seqlens does: the rows that are there are
    written, and that some are missing is reported."""
    T, H, D = 12, 2, 64
    k, v = (rnd(s, T, H, D, dtype=BF).to(DEV) for s in (251, 252))
    w, f = torch.ones(D, device=DEV), gdn.rope_inv_freq(32, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    for fused in (False, True):
        full, cut = (Pool([20, 30], [5, 7], H, D, 16, held, seed=2) for _ in range(2))
        for pool, n in ((full, T), (cut, T - 3)):
            if fused:
                gdn.qk_norm_rope_cache(k[:n], k[:n], v[:n], w, w, pos[:n], f, pool.cache, *pool.where)
            else:
                gdn.kv_cache_write(k[:n], v[:n], pool.cache, *pool.where)
            if pool is cut:
                status_bad()
            gdn.check_device_status(DEV)
        for name in ("k", "v"):
            assert torch.equal(cut.rows(0, range(15, 20), name), full.rows(0, range(15, 20), name))
            assert torch.equal(cut.rows(1, range(23, 27), name), full.rows(1, range(23, 27), name))
            assert (cut.rows(1, range(27, 30), name) == 0).all()
