"""Host-side checks of the softmax-attention layer's calls (no GPU needed):
every C entry point refuses bad arguments before it touches a device, the
binding refuses bad tensors, and the helpers are right."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_silu_b200 as gdn
from gated_deltanet_linear_silu_b200 import build as gbuild
from gated_deltanet_linear_silu_b200.softmax_attention import _CacheStruct

OK, INVALID, UNSUPPORTED, WORKSPACE, NO_DEVICE = 0, 1, 2, 3, 4
A = 1 << 20  # aligned, never dereferenced: validation fails first
B = 1 << 21
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdn.lib()


def cache(**kw):
    a = dict(k=A, v=A, k_scale=A, v_scale=A, n_pages=4, page=16, Hk=2, D=64, dtype=2)
    a.update(kw)
    return ctypes.byref(_CacheStruct(*a.values()))


def pages(**kw):
    a = dict(cache=cache(), table=A, max_pages=2, lens=A, cu=A, N=1)
    a.update({x: y for x, y in kw.items() if x in a})
    return list(a.values())


BAD_CACHE = [
    (dict(n_pages=0), INVALID), (dict(n_pages=-1), INVALID), (dict(Hk=0), INVALID), (dict(k=None), INVALID),
    (dict(v=A + 8), INVALID), (dict(k_scale=None), INVALID), (dict(v_scale=A + 4), INVALID),
    (dict(dtype=0), INVALID), (dict(dtype=3), INVALID), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
    (dict(page=2048), UNSUPPORTED), (dict(page=0), UNSUPPORTED), (dict(page=-16), UNSUPPORTED),
    (dict(D=24), UNSUPPORTED), (dict(D=272), UNSUPPORTED), (dict(D=0), UNSUPPORTED),
]
BAD_PAGES = [(dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(cu=None), INVALID),
             (dict(max_pages=0), INVALID), (dict(max_pages=-1), INVALID), (dict(N=-1), INVALID)]
FROM_PAGES = [(dict(cache=cache(**kw)), st) for kw, st in BAD_CACHE] + [(dict(cache=None), INVALID)] + BAD_PAGES


def norm_rope(L, **kw):
    a = dict(q=A, k=A, dt=1, T=3, H=4, Hk=2, D=64, ldq=0, ldk=0, qw=A, kw=A, eps=1e-6, pos=A, f=A, rot=32, il=0,
             qo=B, ko=2 * B, stream=None)
    a.update(kw)
    return L.gdn_qk_norm_rope(*a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(dt=2), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), UNSUPPORTED), (dict(H=0), INVALID),
    (dict(Hk=0), INVALID), (dict(D=8), UNSUPPORTED), (dict(D=72), UNSUPPORTED), (dict(D=512), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=A + 2), INVALID), (dict(qw=None), INVALID), (dict(kw=None), INVALID),
    (dict(pos=None), INVALID), (dict(f=None), INVALID), (dict(rot=66), INVALID), (dict(rot=-2), INVALID),
    (dict(rot=24), UNSUPPORTED), (dict(il=2), INVALID), (dict(eps=NAN), INVALID), (dict(eps=-1.0), INVALID),
    (dict(ldq=255), INVALID), (dict(ldk=130), INVALID), (dict(qo=None), INVALID), (dict(ko=None), INVALID),
    (dict(qo=A, ldq=512), INVALID), (dict(ko=A, ldk=256), INVALID), (dict(qo=B, ko=B), INVALID),
    (dict(qo=B + 8), INVALID),
])
def test_qk_norm_rope_refuses(L, kw, expect):
    assert norm_rope(L, **kw) == expect


def rope_cache(L, **kw):
    a = dict(q=A, k=A, v=A, dt=1, T=3, H=4, ldq=0, ldk=0, ldv=0, qw=A, kw=A, eps=1e-6, pos=A, f=A, rot=32, il=0)
    a.update({x: y for x, y in kw.items() if x in a})
    return L.gdn_qk_norm_rope_cache(*a.values(), *pages(**kw), kw.get("qo", B), None)


@pytest.mark.parametrize("kw,expect", FROM_PAGES + [
    (dict(dt=2), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), UNSUPPORTED), (dict(N=0), INVALID),
    (dict(v=None), INVALID), (dict(v=A + 8), INVALID), (dict(ldv=8), INVALID), (dict(rot=80), INVALID),
    (dict(H=0), INVALID), (dict(qo=None), INVALID), (dict(qo=A, ldq=512), INVALID), (dict(pos=None), INVALID),
])
def test_qk_norm_rope_cache_refuses(L, kw, expect):
    assert rope_cache(L, **kw) == expect


def write(L, **kw):
    a = dict(k=A, v=A, dt=1, T=3, ldk=0, ldv=0)
    a.update({x: y for x, y in kw.items() if x in a})
    return L.gdn_kv_write(*a.values(), *pages(**kw), None)


@pytest.mark.parametrize("kw,expect", FROM_PAGES + [
    (dict(dt=2), INVALID), (dict(T=-2), INVALID), (dict(k=None), INVALID), (dict(v=A + 4), INVALID),
    (dict(ldk=64), INVALID), (dict(ldv=129), INVALID), (dict(N=0), INVALID),
])
def test_kv_write_refuses(L, kw, expect):
    assert write(L, **kw) == expect


def read(L, **kw):
    a = dict(T=3, dt=1, k=A, v=B)
    a.update({x: y for x, y in kw.items() if x in a})
    return L.gdn_kv_read(*pages(**kw), *a.values(), None)


@pytest.mark.parametrize("kw,expect", FROM_PAGES + [
    (dict(dt=2), INVALID), (dict(T=-1), INVALID), (dict(k=None), INVALID), (dict(v=A), INVALID),
    (dict(v=B + 8), INVALID), (dict(N=0), INVALID),
])
def test_kv_read_refuses(L, kw, expect):
    assert read(L, **kw) == expect


def accept(L, **kw):
    a = dict(path=A, M=4, out=B)
    a.update({x: y for x, y in kw.items() if x in a})
    return L.gdn_kv_accept(*pages(**kw), *a.values(), None)


@pytest.mark.parametrize("kw,expect", FROM_PAGES + [
    (dict(M=-1), INVALID), (dict(M=65), UNSUPPORTED), (dict(path=None), INVALID), (dict(out=None), INVALID),
    (dict(out=A), INVALID),  # the new lengths must not be the old ones
])
def test_kv_accept_refuses(L, kw, expect):
    assert accept(L, **kw) == expect


def attend(L, **kw):
    a = dict(q=A, dt=1, T=3, ldq=0, H=4)
    b = dict(mask=A, nodes=8, scale=0.1, gate=None, o=B, lse=None, ws=A, bytes=1 << 40)
    for x in (a, b):
        x.update({i: y for i, y in kw.items() if i in x})
    return L.gdn_tree_attention(*a.values(), *pages(**kw), *b.values(), None)


@pytest.mark.parametrize("kw,expect", FROM_PAGES + [
    (dict(dt=0), UNSUPPORTED), (dict(dt=2), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID),
    (dict(H=3), INVALID), (dict(H=130), UNSUPPORTED), (dict(cache=cache(n_pages=1 << 27)), UNSUPPORTED), (dict(nodes=0), INVALID), (dict(nodes=65), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(cache=cache(D=96)), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(o=None), INVALID), (dict(o=A), INVALID), (dict(q=A + 8), INVALID), (dict(gate=A + 2), INVALID),
    (dict(gate=B), INVALID), (dict(mask=A + 4), INVALID), (dict(lse=A + 2), INVALID), (dict(ldq=128), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=A + 16), WORKSPACE), (dict(bytes=256), WORKSPACE), (dict(N=0), INVALID),
])
def test_tree_attention_refuses(L, kw, expect):
    assert attend(L, **kw) == expect


def test_too_many_heads(L):
    many = 1 << 17
    assert norm_rope(L, H=many) == UNSUPPORTED and norm_rope(L, Hk=many) == UNSUPPORTED
    assert rope_cache(L, H=many) == UNSUPPORTED
    for call in (rope_cache, write, read, accept, attend):
        assert call(L, cache=cache(Hk=many)) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(H=5), dict(H=130), dict(max_nodes=65), dict(H=0), dict(max_nodes=0), dict(N=-1)])
def test_workspace_size_of_unsupported_arguments(L, kw):
    a = dict(N=1, H=4, max_nodes=2)
    a.update(kw)
    assert L.gdn_tree_attention_workspace_size(cache(), *a.values()) == 0


def at(n):
    """Addresses 16 MB apart, for buffers that share nothing."""
    return n << 24


# a cache of 4 pages of 16 rows of 2 heads of 64: 8192 bytes of values, 512 of scales
APART_CACHE = dict(k=at(10), v=at(11), k_scale=at(12), v_scale=at(13))
# queries [3, 4, 64] bf16: 1536 bytes; keys [3, 2, 64]: 768; fp32 weights 256
APART = dict(cache=cache(**APART_CACHE), table=at(14), lens=at(15), cu=at(16), q=at(1), k=at(2), v=at(3), qw=at(4), kw=at(5),
             pos=at(6), f=at(7), qo=at(8), ko=at(9), path=at(17), out=at(18), mask=at(19), gate=at(20), o=at(21),
             lse=at(22), ws=at(23))


def apart(call, L, **kw):
    a = dict(APART, **({"bytes": 1 << 23} if call is attend else {}), **kw)
    if call is norm_rope:
        for x in ("cache", "table", "lens", "cu", "v", "path", "out", "mask", "gate", "o", "lse", "ws"):
            del a[x]
    if call is read:
        a["k"], a["v"] = kw.get("k", at(24)), kw.get("v", at(25))
    return call(L, **a)


OVERLAPPING = [
    (norm_rope, dict(qo=at(2))), (norm_rope, dict(ko=at(1))), (norm_rope, dict(qo=at(1) + 16)), (norm_rope, dict(qo=at(1) - 16)),
    (norm_rope, dict(ko=at(2) + 752)), (norm_rope, dict(ko=at(8) + 1520)), (norm_rope, dict(ko=at(8) - 752)),
    (norm_rope, dict(ko=at(8))), (norm_rope, dict(qw=at(8) + 1520)), (norm_rope, dict(kw=at(9) + 752)),
    (norm_rope, dict(pos=at(8) + 8)), (norm_rope, dict(f=at(9) - 120)),
    (norm_rope, dict(ldq=4096, qo=at(1) + 16384 - 16 + 512 - 16)),  # rows 8192 bytes apart: the end of the last
    (norm_rope, dict(ldk=4096, qo=at(2) + 8192 - 1520)),            # the start of the second
    (rope_cache, dict(qo=at(2))), (rope_cache, dict(qo=at(3) + 752)), (rope_cache, dict(qo=at(1) + 512)),
    (rope_cache, dict(qo=at(10) + 8176)), (rope_cache, dict(qo=at(13))), (rope_cache, dict(qo=at(14))),
    (rope_cache, dict(q=at(10))), (rope_cache, dict(k=at(11) + 512)), (rope_cache, dict(v=at(12) - 752)),
    (rope_cache, dict(lens=at(10))), (rope_cache, dict(pos=at(8) + 4)),
    (write, dict(k=at(10))), (write, dict(v=at(11) + 8176)), (write, dict(v=at(10) - 752)), (write, dict(table=at(12) + 508)),
    (write, dict(cache=cache(**{**APART_CACHE, "v": at(10)}))), (write, dict(cache=cache(**{**APART_CACHE, "k_scale": at(10)}))),
    (read, dict(k=at(25))), (read, dict(k=at(25) + 752)), (read, dict(v=at(24) + 752)), (read, dict(k=at(10))),
    (read, dict(v=at(13) + 496)), (read, dict(lens=at(24) + 4)),
    (accept, dict(out=at(15))), (accept, dict(out=at(16) + 4)), (accept, dict(out=at(17) + 12)), (accept, dict(out=at(14) + 4)),
    (accept, dict(out=at(10) + 64)), (accept, dict(path=at(11) + 64)), (accept, dict(N=2, out=at(15) + 4)),
    (accept, dict(N=2, out=at(15) - 4)),
    (attend, dict(o=at(1))), (attend, dict(o=at(1) + 1520)), (attend, dict(gate=at(21))), (attend, dict(gate=at(21) - 1520)),
    (attend, dict(mask=at(21) + 8)), (attend, dict(lse=at(21) + 1532)), (attend, dict(lse=at(1))), (attend, dict(lse=at(16))),
    (attend, dict(o=at(11) + 4096)), (attend, dict(ws=at(21))), (attend, dict(ws=at(1))), (attend, dict(ws=at(22))),
    (attend, dict(ws=at(10) - 256)), (attend, dict(lens=at(23) + 512)),
]
BESIDE = [  # what lies right beside, or in place
    (norm_rope, {}), (norm_rope, dict(qo=at(1), ko=at(2))), (norm_rope, dict(qo=at(2) - 1536, ko=at(2))),
    (norm_rope, dict(ldq=4096, qo=at(1) + 512)), (norm_rope, dict(ldq=4096, ko=at(1) + 16384 - 768)),
    (norm_rope, dict(T=1, ko=at(1) + 512)), (norm_rope, dict(T=1, ldq=1024, ko=at(1) + 512)),
    (rope_cache, {}), (rope_cache, dict(qo=at(1))), (rope_cache, dict(k=at(1) + 512, v=at(1) + 768, ldq=512, ldk=512, ldv=512)),
    (write, {}), (write, dict(k=at(3) + 256, ldk=256, ldv=256)), (write, dict(v=at(10) + 8192)), (read, {}),
    (read, dict(k=at(25) - 768)), (accept, {}), (accept, dict(out=at(15) + 4)), (attend, {}), (attend, dict(o=at(1) + 1536)),
    (attend, dict(cache=cache(k=at(10), v=at(10), k_scale=at(12), v_scale=at(12)))), (attend, dict(gate=None, lse=None, mask=None)),
]


@pytest.mark.parametrize("call,kw", OVERLAPPING)
def test_overlapping_buffers_are_refused(L, call, kw):
    assert apart(call, L, **kw) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory: only where no device can run the call")
@pytest.mark.parametrize("call,kw", BESIDE)
def test_buffers_beside_each_other_are_not_refused(L, call, kw):
    assert apart(call, L, **kw) == NO_DEVICE


@pytest.mark.parametrize("kw", [kw for kw, _ in BAD_CACHE if not {"k", "v", "k_scale", "v_scale"} & set(kw)] + [
    dict(dtype=7), dict(n_pages=1 << 27), dict(n_pages=(1 << 31) // 32), dict(D=96), dict(Hk=1 << 17)])
def test_workspace_size_of_unsupported_caches(L, kw):
    """0 for every cache that the attention refuses, whatever its memory."""
    assert L.gdn_tree_attention_workspace_size(cache(**kw), 1, 4 * kw.get("Hk", 2) or 4, 2) == 0
    empty = dict(k=None, v=None, k_scale=None, v_scale=None)
    assert L.gdn_tree_attention_workspace_size(cache(**empty), 1, 4, 2) > 0


def test_workspace_size_of_too_many_units(L):
    size = lambda N: L.gdn_tree_attention_workspace_size(cache(Hk=1 << 16, n_pages=1), N, 1 << 16, 2)
    assert size(1) > 0 and size(1 << 15) == 0


def test_empty_calls_do_nothing(L):
    empty = dict(N=0, table=None, lens=None, cu=None)
    assert norm_rope(L, T=0, q=None, k=None) == OK
    assert rope_cache(L, T=0, q=None, k=None, v=None, **empty) == OK
    assert write(L, T=0, k=None, v=None, **empty) == OK
    assert read(L, T=0, k=None, v=None, **empty) == OK
    assert accept(L, path=None, out=None, **empty) == OK
    assert attend(L, T=0, q=None, o=None, ws=None, **empty) == OK


def test_workspace_size(L):
    size = lambda c, N, H, nodes: L.gdn_tree_attention_workspace_size(c, N, H, nodes)
    assert size(cache(), 4, 8, 8) > 0 and size(cache(), 4, 8, 8) % 256 == 0
    assert size(cache(), 4096, 8, 8) > size(cache(), 4, 8, 8)
    assert size(None, 4, 8, 8) == size(cache(D=96), 4, 8, 8) == size(cache(), 4, 8, 0) == size(cache(), -1, 8, 8) == 0


def test_binding_refuses_tensors(L):
    """What can be seen without a device: shapes, types and host tensors."""
    t = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d)
    f8, f32, i32, f64 = torch.float8_e4m3fn, torch.float32, torch.int32, torch.float64
    with pytest.raises(TypeError):
        gdn.kv_cache(2, 16, 1, 64, dtype=f32, device="cpu")
    q, k, w = t(3, 4, 64), t(3, 2, 64), t(64, d=f32)
    pos, f = t(3, d=i32), t(16, d=f64)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.qk_norm_rope(q, k, w, w, pos, f)
    held = gdn.kv_cache(2, 16, 2, 64, device="cpu")
    pages = (t(1, 2, d=i32), t(1, d=i32), t(2, d=i32))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.qk_norm_rope_cache(q, k, k, w, w, pos, f, held, *pages)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.kv_cache_write(k, k, held, *pages)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.kv_cache_read(held, *pages, n_tokens=3)
    with pytest.raises(TypeError):
        gdn.kv_cache_read(held, *pages, n_tokens=3, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.kv_cache_accept(held, *pages, t(1, 4, d=i32))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.tree_attention(q, held, *pages, max_nodes=3)
    with pytest.raises(TypeError):
        gdn.kv_cache_write(None, k, held, *pages)
    assert f8 == held.k.dtype


@pytest.mark.parametrize("what", ["torch", "abi", "python"])
def test_binding_for_another_torch_or_python_is_stale(L, monkeypatch, what):
    """The binding is compiled against one PyTorch's classes and one Python's: for
    others it is built again, and not loaded before."""
    from gated_deltanet_linear_silu_b200 import softmax_attention

    assert gbuild.binding_up_to_date()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", torch.__version__ + "1")
    elif what == "abi":
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    else:
        import sysconfig
        config = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399" if name == "SOABI" else config(name))
    assert not gbuild.binding_up_to_date()
    monkeypatch.setattr(softmax_attention, "_bound", None)
    with pytest.raises(RuntimeError, match="build"):
        softmax_attention._binding()


def test_tree_mask():
    #   0        0
    #  / \       |
    # 1   2      1      and an empty draft between
    # |
    # 3
    mask, depth = gdn.tree_mask(torch.tensor([-1, 0, 0, 1, -1, 0]), torch.tensor([0, 4, 4, 6]))
    assert mask.tolist() == [0b1, 0b11, 0b101, 0b1011, 0b1, 0b11]
    assert depth.tolist() == [0, 1, 1, 2, 0, 1]
    chain, depth = gdn.tree_mask(torch.arange(-1, 63), torch.tensor([0, 64]))
    assert chain.tolist() == [(1 << i + 1) - 1 for i in range(63)] + [-1] and depth.tolist() == list(range(64))
    for parents, cu in [([0], [0, 1]), ([-1, 1], [0, 2]), ([-2], [0, 1]), ([-1] * 65, [0, 65]), ([-1], [0, 2])]:
        with pytest.raises(ValueError):
            gdn.tree_mask(torch.tensor(parents), torch.tensor(cu))


def test_rope_inv_freq():
    f = gdn.rope_inv_freq(64)
    assert f.dtype == torch.float64 and f.numel() == 32 and f[0] == 1.0
    assert abs(f[16].item() - 1e7 ** -0.5) < 1e-18
