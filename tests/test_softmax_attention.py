"""The softmax-attention layer's kernels against their fp64 restatement
(oracle/attention.py), elementwise.

Tolerances, fixed by arithmetic (u(t) = torch.finfo(t).eps / 2, a rounding's
largest relative error; e = 2^-24 that of fp32):

norm and rotation   y = x inv w: the sum of D <= 256 squares in groups of 8 and
                    5 shuffles (13 e, halved by the root), mean, eps, root,
                    reciprocal, two products: under 13 e. Angle: the turns' cast
                    to fp32 is off by e/2, 2 pi e/2 < 4 e of a radian, sincospi
                    2 ulp each: under 8 e. Products and the sum: 3 e. In all under
                    24 e < 2^-19 of |a| + |b|, then u(t) of the result.
e4m3 rows           scale: the largest element's error / 448 and a division (e).
                    code: half a step, 2^-4 of it or 2^-10 below 2^-6, after a
                    division and the scale's error (under 4 e).
attention           scores: D products and additions, off by D e sum|q||k| scale
                    each way, 2 more scalings; exp2 2 ulp: s = (D + 8) e size + 8 e.
                    A numerator is off by 2 s in total (its own and the total's)
                    and by u(bf16) from its rounding (f16, where the cache is e4m3, is
                    finer); the sums over a row by e for each addition in a chain: no
                    chain is longer than a CTA's stretch, under 2^15 tokens here: 2^-9.
                    Output u(bf16).
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import gated_deltanet_linear_silu_b200 as gdn
from oracle import attention as ref

DEV = torch.device("cuda", 0)
E = 2.0 ** -24
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(DEV)


@pytest.fixture(autouse=True)
def _status():
    """No kernel of a test may have skipped work or given up a wait unnoticed."""
    yield
    gdn.check_device_status(DEV)


def half_step(t):
    return torch.finfo(t).eps / 2


def close(got, want, tol):
    """|got - want| <= tol elementwise, NaN and infinities alike."""
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape
    assert torch.equal(got.isnan(), want.isnan())
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf])
    on = want.isfinite()
    off = (got - want).abs()[on]
    bad = off > tol.expand_as(want)[on]
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {float(off.max()):.3g}"


def rnd(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def status_bad():
    with pytest.raises(gdn.GDNError):
        gdn.check_device_status(DEV)


class Pool:
    """A cache with pages dealt out in shuffled order, and its arguments."""

    def __init__(self, lens, counts, Hk, D, page, dtype, seed=0, spare=1, fill=None):
        need = [-(-l // page) for l in lens]
        P = sum(need) + spare
        order = np.random.default_rng(seed).permutation(P)
        table = np.full((len(lens), max(need + [1]) + 1), -7, np.int32)
        at = 0
        for i, m in enumerate(need):
            table[i, :m] = order[at:at + m]
            at += m
        self.table, self.page, self.ids = torch.from_numpy(table).to(DEV), page, table
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.cu = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
        self.counts, self.host_lens = list(counts), list(lens)
        self.cache = gdn.kv_cache(P, page, Hk, D, dtype=dtype, device=DEV)
        if fill is not None:
            x = rnd(fill, 2, P, Hk, page, D).to(DEV)
            if dtype == BF:
                self.cache.k.copy_(x[0]), self.cache.v.copy_(x[1])
            else:
                for c, s, y in ((self.cache.k, self.cache.k_scale, x[0]), (self.cache.v, self.cache.v_scale, x[1])):
                    s.copy_(y.abs().amax(-1) / 448)
                    c.copy_((y / s[..., None]).to(F8))

    @property
    def where(self):
        return self.table, self.lens, self.cu

    def spots(self, n, positions):
        p = np.atleast_1d(positions)
        return (torch.from_numpy(self.ids[n, p // self.page].astype(np.int64)), torch.from_numpy(p % self.page))

    def rows(self, n, positions, name):
        """fp64 values [len(positions), Hk, D] of the cache's rows, on the host."""
        page, row = self.spots(n, positions)
        x = getattr(self.cache, name).cpu()
        x = x.view(torch.uint8)[page, :, row].view(F8).double() if x.dtype == F8 else x[page, :, row].double()
        s = getattr(self.cache, name + "_scale")
        return x if s is None else x * s.cpu()[page, :, row].double()[..., None]

    def snapshot(self):
        return [None if t is None else (t.view(torch.uint8) if t.dtype == F8 else t).clone() for t in self.cache]


# ---------------------------------------------------------------- norm and rotation

def norm_case(seed, T, H, Hk, D, rotary, dtype, strided, far=2000000):
    wide = rnd(seed, T, (H + 2 * Hk) * D + 16, dtype=dtype).to(DEV)
    parts = [wide[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, H), (H, H + Hk), (H + Hk, H + 2 * Hk))]
    if not strided:
        parts = [p.contiguous() for p in parts]
    w = [1 + 0.1 * rnd(seed + i, D) for i in (1, 2)]
    pos = torch.from_numpy(np.random.default_rng(seed).integers(0, far, T).astype(np.int32))
    return parts, w, pos, gdn.rope_inv_freq(rotary)


def norm_want(x, w, pos, f, eps, il):
    y = ref.norm(x.cpu(), w, eps)
    return ref.rotate(y, pos, f, il), 2.0 ** -19 * ref.pair_size(y, f.numel(), il)


@pytest.mark.parametrize("T,H,Hk,D,rotary,il,dtype,strided", [
    (1, 8, 2, 256, 64, False, BF, True), (5, 3, 1, 128, 128, False, F32, True), (7, 4, 4, 64, 32, True, BF, False),
    (3, 2, 1, 96, 48, False, BF, True), (33, 5, 5, 16, 16, False, F32, False), (9, 1, 1, 48, 0, False, BF, True),
    (2401, 2, 1, 80, 80, True, F32, True), (700, 16, 2, 256, 256, False, BF, True), (64, 7, 7, 240, 16, False, F32, True),
    (2500, 1, 1, 32, 32, False, BF, False),
])
def test_qk_norm_rope(T, H, Hk, D, rotary, il, dtype, strided):
    (q, k, _), w, pos, f = norm_case(11, T, H, Hk, D, rotary, dtype, strided)
    got = gdn.qk_norm_rope(q, k, w[0].to(DEV), w[1].to(DEV), pos.to(DEV), f.to(DEV), interleaved=il, eps=1e-5)
    for g, x, ww in zip(got, (q, k), w):
        want, tol = norm_want(x, ww, pos, f, 1e-5, il)
        assert g.is_contiguous() and g.dtype == dtype
        close(g, want, tol + half_step(dtype) * want.abs())


def test_qk_norm_rope_in_place_and_special_rows():
    (q, k, _), w, pos, f = norm_case(12, 6, 2, 1, 64, 32, BF, False)
    q[1] = 0                      # a zero row stays zero: 0 / sqrt(eps)
    q[2, 0, 3] = float("inf")     # inf / inf in its element, 0 elsewhere
    k[4, 0, 5] = float("nan")     # the whole row
    pos[0] = -17                  # a position below zero turns backwards
    wantq, tolq = norm_want(q, w[0], pos, f, 1e-6, False)
    wantk, tolk = norm_want(k, w[1], pos, f, 1e-6, False)
    a, b = gdn.qk_norm_rope(q, k, w[0].to(DEV), w[1].to(DEV), pos.to(DEV), f.to(DEV), out_q=q, out_k=k)
    assert a is q and b is k
    close(q, wantq, torch.nan_to_num(tolq) + half_step(BF) * torch.nan_to_num(wantq).abs())
    close(k, wantk, torch.nan_to_num(tolk) + half_step(BF) * torch.nan_to_num(wantk).abs())
    (q, k, _), w, pos, f = norm_case(12, 0, 2, 1, 64, 32, BF, False)
    a, b = gdn.qk_norm_rope(q, k, w[0].to(DEV), w[1].to(DEV), pos.to(DEV), f.to(DEV))
    assert a.shape == (0, 2, 64) and b.shape == (0, 1, 64)


def test_qk_norm_rope_refuses_in_place_over_a_view():
    (q, k, _), w, pos, f = norm_case(13, 6, 2, 1, 64, 32, BF, True)
    with pytest.raises(ValueError):
        gdn.qk_norm_rope(q, k, w[0].to(DEV), w[1].to(DEV), pos.to(DEV), f.to(DEV), out_q=q)


# ---------------------------------------------------------------- the cache

def e4m3_tol(x, scale):
    """Bound on |code * scale - x| for a row scaled by `scale` (fp64 [..., 1])."""
    return scale * torch.maximum((x / scale).abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64)) \
        * (1 + 8 * E) + 8 * E * x.abs()


SHAPES = [  # lens, counts, Hk, D, page
    ([1], [1], 1, 64, 16), ([40, 0, 17, 100], [3, 0, 17, 1], 3, 128, 16), ([33, 70], [33, 64], 2, 256, 32),
    ([300, 5, 64], [300, 2, 64], 1, 48, 64), ([130] * 9, [13] * 9, 2, 16, 128),
]


@pytest.mark.parametrize("lens,counts,Hk,D,page", SHAPES)
@pytest.mark.parametrize("dtype,held", [(BF, F8), (F32, F8), (BF, BF), (F32, BF)])
def test_kv_write_and_read(lens, counts, Hk, D, page, dtype, held):
    pool = Pool(lens, counts, Hk, D, page, held, fill=3)
    before = pool.snapshot()
    T = sum(counts)
    pad = 5  # packed rows behind the last sequence
    wide = rnd(5, T + pad, 2 * Hk * D + 8, dtype=dtype).to(DEV)
    k, v = (wide[:, i * Hk * D:(i + 1) * Hk * D].unflatten(1, (Hk, D)) for i in (0, 1))
    gdn.kv_cache_write(k, v, pool.cache, *pool.where)
    gdn.check_device_status(DEV)
    touched = torch.zeros(pool.cache.k.shape[:3], dtype=torch.bool)
    at = 0
    for n, (l, c) in enumerate(zip(lens, counts)):
        if not c:
            continue
        page_, row = pool.spots(n, np.arange(l - c, l))
        touched[page_, :, row] = True
        for name, x in (("k", k), ("v", v)):
            x = x[at:at + c].cpu()
            if held == BF:
                assert torch.equal(getattr(pool.cache, name).cpu()[page_, :, row], x.to(BF))
                continue
            scale = x.float().abs().amax(-1) / 448  # the definition in fp32: the bits agree
            assert torch.equal(getattr(pool.cache, name + "_scale").cpu()[page_, :, row], scale)
            code = (x.float() / scale[..., None]).to(F8)
            assert torch.equal(getattr(pool.cache, name).cpu().view(torch.uint8)[page_, :, row], code.view(torch.uint8))
            got = pool.rows(n, np.arange(l - c, l), name)
            assert ((got - x.double()).abs() <= e4m3_tol(x.double(), scale.double()[..., None])).all()
        at += c
    for t, b in zip(pool.snapshot(), before):  # every other row as it was
        if t is not None:
            assert torch.equal(t.cpu()[~touched], b.cpu()[~touched])
    # read back: the same rows, rounded once; rows behind the last sequence as they were
    for out in (BF, F32):
        ok, ov = (torch.full((T + pad, Hk, D), 7.0, dtype=out, device=DEV) for _ in range(2))
        a, b = gdn.kv_cache_read(pool.cache, *pool.where, n_tokens=T + pad, dtype=out, out_k=ok, out_v=ov)
        gdn.check_device_status(DEV)
        assert (a[T:] == 7).all() and (b[T:] == 7).all()
        at = 0
        for n, (l, c) in enumerate(zip(lens, counts)):
            for name, x in (("k", a), ("v", b)):
                # code * scale is one fp32 product
                want = pool.rows(n, np.arange(l - c, l), name).float().to(out) if c else x[at:at, :, :].cpu()
                assert torch.equal(x[at:at + c].cpu(), want)
            at += c


def test_kv_write_special_rows():
    pool = Pool([8], [8], 1, 32, 16, F8)
    k = rnd(6, 8, 1, 32)
    k[0] = 0
    k[1, 0, 4] = float("inf")
    k[2, 0, 9] = float("nan")
    k[3] = 1e38
    k[4] = 1e-39              # subnormal amax: the scale is subnormal, the codes still of its size
    k[5] = torch.finfo(F32).max
    k[6] = 1e-45              # the scale rounds to zero
    gdn.kv_cache_write(k.to(DEV), k.to(DEV), pool.cache, *pool.where)
    got = pool.rows(0, range(8), "k")
    assert (got[0] == 0).all() and pool.cache.k_scale[pool.ids[0, 0], 0, 0] == 0
    assert got[1].isnan().all() and got[2].isnan().all()
    assert (got[6] == 0).all()
    for i in (3, 5, 7):
        x = k[i].double()
        assert ((got[i] - x).abs() <= e4m3_tol(x, x.abs().max() / 448)).all()
    # 1e-39 / 448 is 1593.1 steps of 2^-149: off by half a step at most, 2^-11 of it
    assert ((got[4] / 1e-39 - 1).abs() <= 2.0 ** -4 + 2.0 ** -11).all()
    codes = pool.cache.k.view(torch.uint8)
    assert not ((codes & 0x7F) == 0x7F).any()  # never an e4m3 NaN
    a, _ = gdn.kv_cache_read(pool.cache, *pool.where, n_tokens=8, dtype=F32)
    assert a[1].isnan().all() and a[2].isnan().all() and (a[0] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("held", [F8, BF])
@pytest.mark.parametrize("T,H,Hk,D,rotary,page", [(1, 8, 2, 256, 64, 64), (23, 3, 3, 128, 32, 16), (2390, 2, 1, 64, 64, 32)])
def test_qk_norm_rope_cache(T, H, Hk, D, rotary, page, held, dtype):
    counts = [T] if T == 1 else [T - 12, 0, 9]  # the last three packed rows belong to nobody
    lens = [T + 50] if T == 1 else [T + 40, 3, 9]
    (q, k, v), w, pos, f = norm_case(21, T, H, Hk, D, rotary, dtype, True)
    pool = Pool(lens, counts, Hk, D, page, held, fill=4)
    other = gdn.KVCache(*[None if t is None else t.clone() for t in pool.cache])
    args = (w[0].to(DEV), w[1].to(DEV), pos.to(DEV), f.to(DEV))
    out = torch.full((T, H, D), 7.0, dtype=dtype, device=DEV)
    got = gdn.qk_norm_rope_cache(q, k, v, *args, pool.cache, *pool.where, out_q=out)
    gdn.check_device_status(DEV)
    m = sum(counts)
    qq, kk = gdn.qk_norm_rope(q, k, *args)
    assert torch.equal(got[:m], qq[:m]) and (got[m:] == 7).all()
    if dtype == F32:  # the two calls one after the other: the same bits
        gdn.kv_cache_write(kk, v, other, *pool.where)
        for a, b in zip(pool.cache, other):
            assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        return
    at = 0
    for n, (l, c) in enumerate(zip(lens, counts)):
        if c:
            want, tol = norm_want(k[at:at + c], w[1], pos[at:at + c], f, 1e-6, False)
            if held == BF:
                close(pool.rows(n, range(l - c, l), "k"), want, tol + half_step(BF) * want.abs())
            else:
                scale = want.abs().amax(-1, keepdim=True) / 448
                lift = tol.amax(-1, keepdim=True) / 448 * 448 * (1 + 2.0 ** -4)  # the scale's error, times a code
                close(pool.rows(n, range(l - c, l), "k"), want, e4m3_tol(want, scale) + tol * (1 + 2.0 ** -4) + lift)
            assert torch.equal(pool.rows(n, range(l - c, l), "v"), _values(v[at:at + c].cpu(), held))
        at += c


def _values(x, held):
    if held == BF:
        return x.to(BF).double()
    s = x.float().abs().amax(-1) / 448
    return (x.float() / s[..., None]).to(F8).double() * s.double()[..., None]


def test_bad_pages_and_bounds_are_skipped():
    """A page id outside the pool, a table too short and a draft longer than its
    sequence: those tokens are skipped and reported, the others are done."""
    k = rnd(8, 40, 1, 32, dtype=BF).to(DEV)
    for what in ("id", "negative", "short", "lens", "cu"):
        pool = Pool([20, 20], [20, 20], 1, 32, 16, BF)
        if what == "id":
            pool.table[0, 1] = pool.cache.k.shape[0]
        elif what == "negative":
            pool.table[0, 1] = -1
        elif what == "short":
            pool.lens[0] = 16 * pool.table.shape[1] + 1
        elif what == "lens":
            pool.lens[0] = 12  # fewer cached than drafted
        else:
            pool.cu[1] = 41
        gdn.kv_cache_write(k, k, pool.cache, *pool.where)
        status_bad()
        gdn.check_device_status(DEV)  # reported once
        if what != "cu":
            assert torch.equal(pool.rows(1, range(20), "k"), k[20:].cpu().double())
        a = torch.full_like(k, 7.0)
        gdn.kv_cache_read(pool.cache, *pool.where, n_tokens=40, out_k=a, out_v=torch.empty_like(k))
        status_bad()
        if what in ("id", "negative"):
            assert torch.equal(a[:16], k[:16]) and (a[16:20] == 7).all() and torch.equal(a[20:], k[20:])


# ---------------------------------------------------------------- accepting

@pytest.mark.parametrize("held", [F8, BF])
@pytest.mark.parametrize("Hk,D,page", [(1, 64, 16), (3, 256, 32), (9, 48, 64)])
def test_kv_accept(held, Hk, D, page):
    lens, counts = [70, 9, 64, 31, 5, 40], [20, 9, 64, 0, 3, 17]
    paths = [[0, 3, 4, 11, 19], [], list(range(64)), [], [2], [0, 1, 2, 9, 10, 11, 12, 13, 14, 15, 16]]
    pool = Pool(lens, counts, Hk, D, page, held, fill=9)
    want = pool.snapshot()
    path = torch.full((6, 64), -1, dtype=torch.int32)
    for n, p in enumerate(paths):
        path[n, :len(p)] = torch.tensor(p, dtype=torch.int32)
        base = lens[n] - counts[n]
        if p:
            src, dst = pool.spots(n, base + np.array(p)), pool.spots(n, base + np.arange(len(p)))
            for t in want:
                if t is not None:
                    moved = t[src[0].to(DEV), :, src[1].to(DEV)].clone()
                    t[dst[0].to(DEV), :, dst[1].to(DEV)] = moved
    got = gdn.kv_cache_accept(pool.cache, *pool.where, path.to(DEV))
    gdn.check_device_status(DEV)
    assert got.tolist() == [l - c + len(p) for l, c, p in zip(lens, counts, paths)] and got.dtype == torch.int32
    for a, b in zip(pool.snapshot(), want):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("path", [[0, 0], [3, 2], [0, 5], [-1, 0], [1, -1, 2]])
def test_kv_accept_refuses_paths(path):
    """Not increasing, outside the draft, or with a gap: nothing moves, the length
    stays, the other sequence is done."""
    pool = Pool([20, 20], [5, 5], 1, 32, 16, F8, fill=2)
    want = pool.snapshot()
    rows = torch.full((2, 4), -1, dtype=torch.int32)
    rows[0, :len(path)] = torch.tensor(path, dtype=torch.int32)
    got = gdn.kv_cache_accept(pool.cache, *pool.where, rows.to(DEV))
    status_bad()
    assert got.tolist() == [20, 15]
    for a, b in zip(pool.snapshot(), want):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- attention

def trees(counts, seed, empty=()):
    g = np.random.default_rng(seed)
    parents = [int(g.integers(-1, i)) if i else -1 for c in counts for i in range(c)]
    mask, _ = gdn.tree_mask(torch.tensor(parents, dtype=torch.int64), torch.tensor([0] + list(np.cumsum(counts))))
    for t in empty:
        mask[t] = 0
    return mask


def check_attention(pool, q, o, lse, mask, scale, gate=None, rows=None):
    at = 0
    D = q.shape[2]
    for n, (l, c) in enumerate(zip(pool.host_lens, pool.counts)):
        if c and (rows is None or n in rows):
            k, v = pool.rows(n, range(l), "k"), pool.rows(n, range(l), "v")
            m = mask[at:at + c] if mask is not None else [(2 << i) - 1 for i in range(c)]
            want, z, mass, size = ref.attention(q[at:at + c].cpu(), k, v, l - c, m, scale,
                                                None if gate is None else gate[at:at + c].cpu())
            s = ((D + 8) * E * size + 8 * E)[..., None]
            u = half_step(BF)
            close(o[at:at + c], want, (u + 2 * s + 2.0 ** -9) * mass * (1 + u) + u * want.abs() + 8 * E * mass)
            close(lse[at:at + c], z, s[..., 0] + 2.0 ** -9 + 8 * E * z.abs().nan_to_num(posinf=0))
        at += c


ATTEND = [  # lens, counts, H, Hk, D, page
    ([1], [1], 1, 1, 64, 16),
    ([15, 16, 17, 64, 65], [1, 1, 1, 1, 1], 4, 2, 128, 16),
    ([700], [1], 8, 2, 256, 64),
    ([33, 0, 5, 260], [9, 0, 5, 3], 6, 2, 64, 32),
    ([64, 130, 64], [64, 64, 63], 4, 1, 128, 16),
    ([90, 1500], [17, 2], 8, 2, 256, 128),
    ([3000, 1, 2, 3], [5, 1, 2, 3], 16, 1, 64, 1024),
    ([513, 40], [16, 33], 3, 3, 128, 64),
    ([200, 77], [64, 31], 64, 1, 64, 16),
    ([211], [50], 10, 2, 256, 16),
]


@pytest.mark.parametrize("lens,counts,H,Hk,D,page", ATTEND)
@pytest.mark.parametrize("held", [F8, BF])
@pytest.mark.parametrize("form", ["chain", "tree"])
@pytest.mark.parametrize("most", ["tight", "loose"])  # max_nodes: the largest draft, or 64
def test_tree_attention(lens, counts, H, Hk, D, page, held, form, most):
    pool = Pool(lens, counts, Hk, D, page, held, fill=31)
    T = sum(counts)
    wide = rnd(32, T, H * D + 8, dtype=BF, scale=1.5).to(DEV)
    q = wide[:, :H * D].unflatten(1, (H, D))
    mask = trees(counts, 5) if form == "tree" else None
    gate = rnd(33, T, H, D, dtype=BF).to(DEV) if form == "tree" else None
    o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=max(counts) if most == "tight" else 64,
                                mask=None if mask is None else mask.to(DEV),
                                gate=gate, return_lse=True)
    gdn.check_device_status(DEV)
    check_attention(pool, q, o, lse, mask, D ** -0.5, gate)


@pytest.mark.parametrize("held", [F8, BF])
@pytest.mark.parametrize("D", [64, 256])
def test_tree_attention_empty_rows_and_padding(held, D):
    """Rows whose mask leaves nothing are zero with lse -inf; a mask without the
    node's own bit, and bits past the draft, which mean nothing; packed rows
    behind the last sequence are left as they were."""
    pool = Pool([6, 40, 3], [6, 9, 3], 2, D, 16, held, fill=41)
    T = 18
    q = rnd(42, T + 4, 4, D, dtype=BF).to(DEV)
    mask = trees([6, 9, 3], 6, empty=[0, 4, 8, 17])
    mask[5] = 0b10 | -(1 << 40)
    pad = torch.cat([mask, torch.full((4,), -1)]).to(DEV)
    out = torch.full((T + 4, 4, D), 7.0, dtype=BF, device=DEV)
    o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=9, mask=pad, out=out, return_lse=True)
    gdn.check_device_status(DEV)
    assert (o[T:] == 7).all()
    for t in (0, 4, 17):
        assert (o[t] == 0).all() and (lse[t] == -math.inf).all()
    check_attention(pool, q, o, lse, [int(m) & 0x1FF for m in mask], D ** -0.5)


@pytest.mark.parametrize("held", [F8, BF])
@pytest.mark.parametrize("lens", [[40], [5000]])
def test_tree_attention_non_finite_behind_the_mask(held, lens):
    """NaN and infinities in a node that a row does not see do not reach it; in
    one that it sees, they do. Rows behind the sequence hold NaN as well."""
    c, D = 8, 128
    pool = Pool(lens, [c], 1, D, 16, held, fill=51)
    base = lens[0] - c
    # node 1: values NaN; node 2: keys NaN; node 3 (bf16): a value +inf in one element
    def put(name, node, value, element=None):
        page, row = (int(x) for x in pool.spots(0, base + node))
        if held == F8:
            getattr(pool.cache, name + "_scale")[page, :, row] = value
        else:
            getattr(pool.cache, name)[page, :, row, slice(None) if element is None else element] = value
    put("v", 1, math.nan)
    put("k", 2, math.nan)
    if held == BF:
        put("v", 3, math.inf, 77)
    tail = lens[0] % 16
    if tail:  # the rest of the last page
        page = pool.ids[0, lens[0] // 16]
        for name in ("k", "v"):
            if held == F8:
                getattr(pool.cache, name + "_scale")[page, :, tail:] = math.nan
                getattr(pool.cache, name).view(torch.uint8)[page, :, tail:] = 0x7F
            else:
                getattr(pool.cache, name)[page, :, tail:] = math.nan
    q = rnd(52, c, 2, D, dtype=BF).to(DEV)
    mask = torch.tensor([0b1, 0b11, 0b101, 0b1001, 0b10001, 0b110001, 0b1010001, 0b10111001], dtype=torch.int64)
    o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=c, mask=mask.to(DEV), return_lse=True)
    gdn.check_device_status(DEV)
    assert o[1].isnan().all() and lse[1].isfinite().all()
    assert o[2].isnan().all() and lse[2].isnan().all()
    for t in ([0, 4, 5, 6] if held == BF else [0, 3, 4, 5, 6, 7]):
        assert o[t].isfinite().all() and lse[t].isfinite().all()
    if held == BF:
        for t in (3, 7):
            assert (o[t, :, 77] == math.inf).all() and o[t, :, :77].isfinite().all() and o[t, :, 78:].isfinite().all()
            assert lse[t].isfinite().all()


@pytest.mark.parametrize("held", [F8, BF])
def test_tree_attention_extreme_scores(held):
    """Scores of the type's lowest and largest size: one key takes all, or, with
    keys at minus infinity, none does."""
    pool = Pool([300], [2], 1, 64, 16, held, fill=61)
    q = rnd(62, 2, 2, 64, dtype=BF, scale=300.0).to(DEV)
    o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=2, scale=30.0, return_lse=True)
    k, v = pool.rows(0, range(300), "k"), pool.rows(0, range(300), "v")
    want, z, mass, size = ref.attention(q.cpu(), k, v, 298, [1, 3], 30.0)
    assert o.isfinite().all() and (lse.cpu().double() - z).abs().max() <= float(80 * E * size.max())
    if held == BF:  # every key -inf in one element: all scores -inf or NaN-free zero rows
        pool.cache.k[:] = 0
        pool.cache.k[..., 0] = -math.inf
        q = torch.zeros(2, 2, 64, dtype=BF, device=DEV)
        q[..., 0] = 1
        o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=2, return_lse=True)
        assert (o == 0).all() and (lse == -math.inf).all()


def test_tree_attention_many_sequences():
    """More sequences than a block scans at once, most of them empty or short."""
    g = np.random.default_rng(7)
    counts = [int(x) for x in g.choice([0, 1, 2, 7], 333)]
    lens = [c + int(g.integers(0, 90)) for c in counts]
    pool = Pool(lens, counts, 1, 64, 16, F8, fill=71)
    q = rnd(72, sum(counts), 2, 64, dtype=BF).to(DEV)
    mask = trees(counts, 8)
    o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=7, mask=mask.to(DEV), return_lse=True)
    gdn.check_device_status(DEV)
    check_attention(pool, q, o, lse, mask, 0.125, rows=range(0, 333, 7))
    empty = Pool([4, 9], [0, 0], 1, 64, 16, F8)
    assert gdn.tree_attention(q[:0], empty.cache, *empty.where, max_nodes=1).shape == (0, 2, 64)


@pytest.mark.parametrize("held", [F8, BF])
def test_tree_attention_long(held):
    """One long sequence, split over the whole GPU and joined."""
    pool = Pool([20000, 9000], [3, 1], 1, 128, 64, held, fill=81)
    q = rnd(82, 4, 4, 128, dtype=BF).to(DEV)
    mask = trees([3, 1], 9)
    o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=3, mask=mask.to(DEV), return_lse=True)
    check_attention(pool, q, o, lse, mask, 128 ** -0.5)
    for _ in range(3):  # the same bits at every call
        again, lse2 = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=3, mask=mask.to(DEV), return_lse=True)
        assert torch.equal(o, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("held", [F8, BF])
@pytest.mark.parametrize("D,nodes", [(64, 1), (64, 9), (128, 1), (128, 5), (256, 1), (256, 3), (256, 6)])
def test_tree_attention_of_one_sequence(held, D, nodes):
    """One sequence alone: a few tiles for each of many CTAs, tens of partials to
    a row, with the gate."""
    pool = Pool([2500], [nodes], 2, D, 32, held, fill=85)
    q, gate = (rnd(s, nodes, 8, D, dtype=BF).to(DEV) for s in (86, 87))
    mask = trees([nodes], 11)
    o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=nodes, mask=mask.to(DEV), gate=gate, return_lse=True)
    check_attention(pool, q, o, lse, mask, D ** -0.5, gate=gate)


@pytest.mark.parametrize("N,nodes", [(128, 1), (129, 1), (300, 2), (512, 9), (513, 9), (700, 9)])
def test_tree_attention_of_many_sequences(N, nodes):
    """More sequences than a CTA has threads, and as many; empty ones among them."""
    g = torch.Generator().manual_seed(N)
    counts = [min(int(c), nodes) for c in torch.randint(0, nodes + 1, (N,), generator=g)]
    lens = [c + int(x) for c, x in zip(counts, torch.randint(0, 70, (N,), generator=g))]
    pool = Pool(lens, counts, 1, 64, 16, F8, fill=88)
    q = rnd(89, sum(counts), 2, 64, dtype=BF).to(DEV)
    o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=nodes, return_lse=True)
    check_attention(pool, q, o, lse, None, 64 ** -0.5)


@pytest.mark.parametrize("held", [F8, BF])
@pytest.mark.parametrize("D,G,nodes", [(64, 8, 40), (128, 4, 7), (256, 4, 17), (128, 16, 20)])
def test_tree_attention_long_with_many_rows(held, D, G, nodes):
    """The same with more rows than one group of eight or sixteen: hundreds of
    tiles to a CTA, several row tiles, one short sequence beside the long one."""
    lens, counts = [120000, 700], [nodes, 3]
    pool = Pool(lens, counts, 2, D, 64, held, fill=83)
    q = rnd(84, sum(counts), 2 * G, D, dtype=BF).to(DEV)
    mask = trees(counts, 10)
    o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=nodes, mask=mask.to(DEV), return_lse=True)
    # the reference on some rows: nodes 0 and the last, every head
    k, v = (pool.rows(0, range(lens[0]), name) for name in ("k", "v"))
    base = lens[0] - nodes
    for i in (0, nodes - 1):
        seen = torch.tensor([j < base or bool(int(mask[i]) >> (j - base) & 1) for j in range(lens[0])])
        for h in (0, G - 1, 2 * G - 1):
            s = (k[:, h // G] @ q[i, h].cpu().double()) * D ** -0.5
            s[~seen] = -math.inf
            z = torch.logsumexp(s, 0)
            p = torch.exp(s - z)
            size = (k[:, h // G].abs() @ q[i, h].cpu().double().abs()).max() * D ** -0.5
            want, mass = p @ v[:, h // G], p @ v[:, h // G].abs()
            e = float((D + 8) * E * size + 8 * E)
            u = half_step(BF)
            close(o[i, h], want, (u + 2 * e + 2.0 ** -9) * mass * (1 + u) + u * want.abs())
            assert abs(float(lse[i, h]) - float(z)) <= e + 2.0 ** -9 + 8 * E * abs(float(z))
    check_attention(pool, q, o, lse, mask, D ** -0.5, rows=[1])


def test_tree_attention_bad_sequences():
    """A draft past max_nodes, a length past the table and a missing page are
    reported; the other sequences are done."""
    for what in ("nodes", "short", "page"):
        pool = Pool([50, 60], [5, 3], 1, 64, 16, F8, fill=91)
        q = rnd(92, 8, 1, 64, dtype=BF).to(DEV)
        if what == "short":
            pool.lens[0] = 1000
        if what == "page":
            pool.table[0, 1] = 1 << 20
        out = torch.full((8, 1, 64), 7.0, dtype=BF, device=DEV)
        o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=4 if what == "nodes" else 8, out=out,
                                    return_lse=True)
        status_bad()
        if what != "page":
            assert (o[:5] == 7).all()
        check_attention(pool, q, o, lse, None, 0.125, rows=[1])


def test_cache_past_32_bits():
    """Rows whose byte and element offsets pass 2^32."""
    P, page, Hk, D = 18000, 128, 8, 256
    cache = gdn.KVCache(*(torch.empty((P, Hk, page, D), dtype=F8, device=DEV) for _ in range(2)),
                        *(torch.empty((P, Hk, page), dtype=F32, device=DEV) for _ in range(2)))
    assert cache.k.numel() > 1 << 32
    table = torch.tensor([[P - 1, 3, P - 2]], dtype=torch.int32, device=DEV)
    lens, cu = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([300], [0, 300]))
    k, v = (rnd(s, 300, Hk, D, dtype=BF) for s in (101, 102))
    gdn.kv_cache_write(k.to(DEV), v.to(DEV), cache, table, lens, cu)
    a, b = gdn.kv_cache_read(cache, table, lens, cu, n_tokens=300, dtype=F32)
    assert torch.equal(a.cpu().double(), _values(k, F8).float().double())
    assert torch.equal(b.cpu().double(), _values(v, F8).float().double())
    q = rnd(103, 2, Hk, D, dtype=BF).to(DEV)
    two = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    o = gdn.tree_attention(q, cache, table, lens, two, max_nodes=2)
    want, z, mass, size = ref.attention(q.cpu(), _values(k, F8), _values(v, F8), 298, [1, 3], D ** -0.5)
    s = ((D + 8) * E * size + 8 * E)[..., None]
    u = half_step(BF)
    close(o, want, (u + 2 * s + 2.0 ** -9) * mass + u * want.abs())
    path = torch.tensor([[0, 150, 299]], dtype=torch.int32, device=DEV)
    assert gdn.kv_cache_accept(cache, table, lens, cu, path).tolist() == [3]
    a, _ = gdn.kv_cache_read(cache, table, torch.tensor([3], dtype=torch.int32, device=DEV),
                             torch.tensor([0, 3], dtype=torch.int32, device=DEV), n_tokens=3, dtype=F32)
    assert torch.equal(a.cpu().double(), _values(k[[0, 150, 299]], F8).float().double())
    gdn.check_device_status(DEV)


# ---------------------------------------------------------------- tensors that are refused

def test_refused_tensors():
    """Shapes, types, strides and devices that the C ABI cannot see."""
    z = lambda *s, d=BF, dev=DEV: torch.zeros(s, dtype=d, device=dev)
    i32, f64 = torch.int32, torch.float64
    q, k, w, pos, f = z(3, 4, 64), z(3, 2, 64), z(64, d=F32), z(3, d=i32), z(16, d=f64)
    ok = [q, k, w, w, pos, f]
    gdn.qk_norm_rope(*ok)
    bad = [(1, z(2, 2, 64)), (1, z(3, 2, 32)), (1, k.float()), (2, w.double()), (2, z(32, d=F32)), (4, pos.long()),
           (4, z(4, d=i32)), (5, f.float()), (5, z(33, d=f64)), (0, q[0]), (2, w.cpu()), (4, z(6, d=i32)[::2]),
           (0, z(3, 4, 128)[..., ::2]), (0, z(3, 64, 4).transpose(1, 2))]
    for i, x in bad:
        args = list(ok)
        args[i] = x
        with pytest.raises((ValueError, TypeError)):
            gdn.qk_norm_rope(*args)
    with pytest.raises(TypeError):
        gdn.qk_norm_rope(q.half(), k.half(), w, w, pos, f)
    with pytest.raises(ValueError):
        gdn.qk_norm_rope(*ok, out_q=z(3, 4, 64, d=F32))
    pool = Pool([20], [3], 2, 64, 16, F8)
    c, pages = pool.cache, pool.where
    gdn.kv_cache_write(k, k, c, *pages)
    for held in (c._replace(v=z(*c.k.shape)), c._replace(k_scale=None), c._replace(v_scale=c.v_scale.double()),
                 c._replace(k_scale=c.k_scale[..., :8]), c._replace(k=c.k.cpu(), v=c.v.cpu()),
                 gdn.KVCache(z(2, 2, 16, 64, d=F32), z(2, 2, 16, 64, d=F32)), c._replace(k=c.k[0], v=c.v[0])):
        with pytest.raises((ValueError, TypeError)):
            gdn.kv_cache_write(k, k, held, *pages)
    for p in ((pages[0].long(), *pages[1:]), (pages[0][0], *pages[1:]), (pages[0], pages[1].repeat(2), pages[2]),
              (pages[0], pages[1], pages[2][:0]), (pages[0].cpu(), *pages[1:]), (pages[0].repeat(2, 1), *pages[1:])):
        with pytest.raises((ValueError, TypeError)):
            gdn.kv_cache_write(k, k, c, *p)
    for a, b in ((k, z(3, 1, 64)), (z(3, 1, 64), z(3, 1, 64)), (k, k.float()), (k[0], k[0])):
        with pytest.raises(ValueError):
            gdn.kv_cache_write(a, b, c, *pages)
    with pytest.raises(ValueError):
        gdn.kv_cache_read(c, *pages, n_tokens=-1)
    with pytest.raises(ValueError):
        gdn.kv_cache_read(c, *pages, n_tokens=3, out_k=z(4, 2, 64))
    with pytest.raises(ValueError):
        gdn.kv_cache_accept(c, *pages, z(2, 4, d=i32))
    with pytest.raises(gdn.GDNError):
        gdn.kv_cache_accept(c, *pages, z(1, 4, d=i32), out_seq_lens=pages[1])
    with pytest.raises(ValueError):
        gdn.tree_attention(z(3, 4, 128), c, *pages, max_nodes=3)
    with pytest.raises(gdn.GDNError):
        gdn.tree_attention(z(3, 3, 64), c, *pages, max_nodes=3)
    with pytest.raises(gdn.GDNError):
        gdn.tree_attention(q.float(), c, *pages, max_nodes=3)
    for kw in (dict(mask=z(2, d=torch.int64)), dict(mask=pos), dict(gate=z(3, 4, 64, d=F32)), dict(out=z(3, 2, 64)),
               dict(workspace=z(64, d=torch.uint8)[::2])):
        with pytest.raises(ValueError):
            gdn.tree_attention(q, c, *pages, max_nodes=3, **kw)
    gdn.check_device_status(DEV)


# ---------------------------------------------------------------- as a serving loop runs them

def test_streams_graphs_and_workspaces():
    """The same results on another stream, from a captured graph replayed with
    new inputs, and from two graphs with a workspace each, replayed at once."""
    pool = Pool([900, 100, 2000], [4, 1, 6], 2, 128, 32, F8, fill=111)
    q = rnd(112, 11, 8, 128, dtype=BF).to(DEV)
    q2 = rnd(113, 11, 8, 128, dtype=BF).to(DEV)
    want, want2 = (gdn.tree_attention(x, pool.cache, *pool.where, max_nodes=6) for x in (q, q2))
    torch.cuda.synchronize()
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        got = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=6)
    side.synchronize()
    assert torch.equal(got, want)
    size = gdn.tree_attention_workspace_size(pool.cache, 3, 8, 6)
    runs = []
    for x in (q.clone(), q2.clone()):
        ws = torch.empty(size, dtype=torch.uint8, device=DEV)
        out = torch.empty_like(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gdn.tree_attention(x, pool.cache, *pool.where, max_nodes=6, out=out, workspace=ws)
        runs.append((graph, x, out, ws, torch.cuda.Stream(DEV)))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, _, _, _, s in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(runs[0][2], want) and torch.equal(runs[1][2], want2)
    runs[0][1].copy_(q2)
    runs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(runs[0][2], want2)
    with pytest.raises(gdn.GDNError):
        gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=6, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("rows", [4, 24])  # query rows: either kernel
def test_inputs_written_just_before(rows):
    """Lengths, queries and pages that the kernel before the call writes, on the
    same stream and behind a long kernel: no part of a call may read them early."""
    pool = Pool([4000, 300], [1, 1], 1, 64, 16, F8, fill=121)
    q = torch.empty(2, rows, 64, dtype=BF, device=DEV)
    qs = [rnd(122 + i, 2, rows, 64, dtype=BF).to(DEV) for i in range(4)]
    lens = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([4000, 300], [17, 290], [3001, 1], [1, 299])]
    table = pool.table.clone()
    want = [gdn.tree_attention(x, pool.cache, table, l, pool.cu, max_nodes=1, return_lse=True) for x, l in zip(qs, lens)]
    big = torch.randn(4096, 4096, device=DEV)
    moving, pages = torch.empty_like(lens[0]), torch.empty_like(table)
    for i in [0, 1, 2, 3] * 6:
        big @ big
        moving.copy_(lens[i])
        pages.copy_(table)
        q.copy_(qs[i])
        o, lse = gdn.tree_attention(q, pool.cache, pages, moving, pool.cu, max_nodes=1, return_lse=True)
        moving.zero_()  # and nothing reads them late
        pages.fill_(-1)
        q.zero_()
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
    # lengths straight from the call that accepts a draft
    for i in range(8):
        new = gdn.kv_cache_accept(pool.cache, table, lens[0], torch.tensor([0, 0, 0], dtype=torch.int32, device=DEV),
                                  torch.empty((2, 0), dtype=torch.int32, device=DEV))
        o = gdn.tree_attention(qs[0], pool.cache, table, new, pool.cu, max_nodes=1)
        assert torch.equal(o, want[0][0])


@pytest.mark.parametrize("held", [F8, BF])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_waits_that_run_out_are_reported(D, held):
    """With the limit at 0 every wait that is not over at its first probe gives up:
    the kernel reports it, frees what it holds, and the next call is right."""
    pool = Pool([3000, 100], [9, 2], 2, D, 32, held, fill=131)
    q = rnd(132, 11, 8, D, dtype=BF).to(DEV)
    gdn.set_wait_limit_ns(0)
    try:
        gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=9)
        with pytest.raises(gdn.GDNError, match="TIMEOUT"):
            gdn.check_device_status(DEV)
    finally:
        gdn.set_wait_limit_ns(-1)
    torch.cuda.synchronize()
    o, lse = gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=9, return_lse=True)
    check_attention(pool, q, o, lse, None, D ** -0.5)


@pytest.mark.parametrize("word", [-1, 0x7FFFFFFF, -0x80000000, 0x7FFFFFFF - (1 << 32) * 0x80000000])
def test_waits_that_run_out_leave_the_workspace_unread(word):
    """Where the first kernel gave up before it noted where its partials are, the
    words that were there mean nothing to the one that adds them up."""
    pool = Pool([3000, 100], [9, 2], 2, 128, 32, F8, fill=133)
    q = rnd(134, 11, 8, 128, dtype=BF).to(DEV)
    size = gdn.tree_attention_workspace_size(pool.cache, 2, 8, 9)
    ws = torch.full((size // 8,), word, dtype=torch.int64, device=DEV).view(torch.uint8)
    gdn.set_wait_limit_ns(0)
    try:
        gdn.tree_attention(q, pool.cache, *pool.where, max_nodes=9, workspace=ws)
        with pytest.raises(gdn.GDNError, match="TIMEOUT"):
            gdn.check_device_status(DEV)
    finally:
        gdn.set_wait_limit_ns(-1)
    torch.cuda.synchronize()


@pytest.mark.parametrize("held", [F8, BF])
def test_drafted_decoding_equals_plain_decoding(held):
    """Prompts, then rounds of drafting, verifying and accepting, captured steps
    and all: the cache holds, bit for bit, what writing the accepted tokens one
    after the other leaves, and each node's attention is that of its path alone,
    decoded plainly."""
    H, Hk, D, page, rotary = 8, 2, 256, 32, 64
    prompts, rounds = [37, 1, 64], 3
    parents = [[-1, 0, 0, 1, 2, 2], [-1, 0], [-1, 0, 1, 2, 0]]
    room = [p + 40 for p in prompts]
    g = torch.Generator().manual_seed(5)
    w = [(1 + 0.1 * torch.randn(D, generator=g)).to(DEV) for _ in range(2)]
    f = gdn.rope_inv_freq(rotary, device=DEV)
    spec, plain = (Pool(room, [1] * 3, Hk, D, page, held, seed=s) for s in (1, 2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)

    def rows(n):
        return [torch.randn((n, h, D), generator=g).to(BF).to(DEV) for h in (H, Hk, Hk)]

    def step(pool, x, pos, lens, cu, nodes, mask=None):
        q = gdn.qk_norm_rope_cache(*x, *w, i32(pos), f, pool.cache, pool.table, lens, cu)
        return gdn.tree_attention(q, pool.cache, pool.table, lens, cu, max_nodes=nodes, mask=mask)

    x = rows(sum(prompts))
    cu = i32([0] + list(np.cumsum(prompts)))
    pos = [p for n in prompts for p in range(n)]
    for pool in (spec, plain):
        gdn.qk_norm_rope_cache(*x, *w, i32(pos), f, pool.cache, pool.table, i32(prompts), cu)
    lens = list(prompts)
    for r in range(rounds):
        counts = [len(p) for p in parents]
        cu = [0] + list(np.cumsum(counts))
        mask, depth = gdn.tree_mask(torch.tensor([p for t in parents for p in t]), torch.tensor(cu))
        drafted = rows(sum(counts))
        full = [l + c for l, c in zip(lens, counts)]
        pos = [lens[n] + int(depth[cu[n] + i]) for n in range(3) for i in range(counts[n])]
        o = step(spec, drafted, pos, i32(full), i32(cu), 6, mask.to(DEV))
        # the deepest path of each tree is accepted on even rounds, the root alone on odd ones
        path = []
        for n, t in enumerate(parents):
            node = max(range(len(t)), key=lambda i: (int(depth[cu[n] + i]), i)) if r % 2 == 0 else 0
            chain = []
            while node >= 0:
                chain.insert(0, node)
                node = t[node]
            path.append(chain)
        kept = torch.full((3, 6), -1, dtype=torch.int32)
        for n, p in enumerate(path):
            kept[n, :len(p)] = torch.tensor(p, dtype=torch.int32)
        new = gdn.kv_cache_accept(spec.cache, spec.table, i32(full), i32(cu), kept.to(DEV))
        # plainly: the accepted tokens of each sequence, one decode step after the other
        for n, p in enumerate(path):
            for a, node in enumerate(p):
                t = cu[n] + node
                one = [y[t:t + 1].contiguous() for y in drafted]
                want = step(_only(plain, n), one, [lens[n] + a], i32([lens[n] + a + 1]), i32([0, 1]), 1)
                # the same sums over the same rows, cut differently: both within the bound of the exact result
                k, v = (plain.rows(n, range(lens[n] + a + 1), name) for name in ("k", "v"))
                qq = gdn.qk_norm_rope(one[0], one[1], *w, i32([lens[n] + a]), f)[0].cpu()
                exact, _, mass, size = ref.attention(qq, k, v, lens[n] + a, [1], D ** -0.5)
                s = ((D + 8) * E * size + 8 * E)[..., None]
                tol = (half_step(BF) + 2 * s + 2.0 ** -9) * mass * (1 + half_step(BF)) + half_step(BF) * exact.abs()
                close(o[t:t + 1], exact, tol)
                close(want, exact, tol)
            lens[n] += len(p)
        assert new.tolist() == lens
        for n in range(3):
            for name in ("k", "v"):
                assert torch.equal(spec.rows(n, range(lens[n]), name), plain.rows(n, range(lens[n]), name))
    gdn.check_device_status(DEV)


class _only:
    """One sequence of a pool."""

    def __init__(self, pool, n):
        self.cache, self.table = pool.cache, pool.table[n:n + 1].contiguous()
