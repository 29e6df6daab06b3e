"""Measured operators of the hybrid model's softmax-attention layers: their plain forms in torch
and the calls of this framework that compute the same.

Five operators over one paged key/value cache (pages [P, Hk, page, D], values in e4m3 with one
fp32 scale per (token, head), or in bf16):

  rope     RMSNorm of each query and key head and the rotation by position, in one pass; with a
           cache the keys and values are quantised and written in the same pass
  write    quantising keys and values as they are written to the cache
  read     reading the cache back as dense keys and values
  accept   moving the accepted nodes of a drafted tree to the front of its cache rows
  attend   attention of a tree of drafted tokens (one node: a plain decode step) over the cache

In every call sequence n's tokens cu_seqlens[n]..cu_seqlens[n+1] stand at the last positions of
its seq_lens[n] cached ones.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token of the 0.8B model's attention layer (8 q heads on 2 kv heads of 256, a
        # quarter of them rotated), far into its context: a pure latency call
        dict(name="rope_decode", op="rope", cache="e4m3", type="bf16", seqs=1, tokens=1, ctx=30011,
             heads=8, kv_heads=2, dim=256, rotary=64, interleaved=False, page=64),
        # a long prompt through the same layer, queries and keys kept as tensors
        dict(name="rope_prefill", op="rope", cache="none", type="bf16", seqs=1, tokens=16384, ctx=16384,
             heads=8, kv_heads=2, dim=256, rotary=64, interleaved=False, page=64),
        # the new token of each of 64 sequences written to an unquantised cache from fp32 activations
        dict(name="write_step", op="write", cache="bf16", type="f32", seqs=64, tokens=64, ctx=4096,
             kv_heads=8, dim=128, page=16),
        # ragged prompts quantised into the cache
        dict(name="write_prefill", op="write", cache="e4m3", type="bf16", seqs=8, tokens=32771, ctx=8192,
             kv_heads=8, dim=128, page=32),
        # a prompt's unquantised keys and values for a kernel that wants them dense
        dict(name="read_one", op="read", cache="bf16", type="f32", seqs=1, tokens=1021, ctx=1021,
             kv_heads=2, dim=256, page=64),
        # the whole quantised cache of a ragged batch read back
        dict(name="read_batch", op="read", cache="e4m3", type="bf16", seqs=64, tokens=131101, ctx=4096,
             kv_heads=8, dim=128, page=16),
        # the accepted path of one 64-node draft
        dict(name="accept_one", op="accept", cache="e4m3", seqs=1, nodes=64, ctx=2049, kv_heads=2,
             dim=256, page=64),
        # the accepted paths of a batch of 24-node drafts
        dict(name="accept_batch", op="accept", cache="bf16", seqs=256, nodes=24, ctx=1024, kv_heads=8,
             dim=128, page=16),
        # one decoded token of one sequence, output gated as in the 0.8B layer: latency
        dict(name="attend_one", op="attend", cache="e4m3", seqs=1, nodes=1, ctx=1021, ragged=False,
             heads=8, kv_heads=2, dim=256, page=64, gate=True),
        # an ordinary decode step of a full batch
        dict(name="attend_batch", op="attend", cache="e4m3", seqs=64, nodes=1, ctx=8192, ragged=False,
             heads=32, kv_heads=8, dim=128, page=64, gate=False),
        # ragged contexts and ragged drafts on the 0.8B layer
        dict(name="attend_ragged", op="attend", cache="e4m3", seqs=24, nodes=17, ctx=16389, ragged=True,
             heads=8, kv_heads=2, dim=256, page=32, gate=True),
        # the largest drafts on long contexts, unquantised cache
        dict(name="attend_large", op="attend", cache="bf16", seqs=8, nodes=64, ctx=32768, ragged=False,
             heads=32, kv_heads=8, dim=128, page=128, gate=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "accept", "attend", "attend"])
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["e4m3", "e4m3", "bf16"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    room = 1024 // (kv_heads * dim // 64)  # fewer tokens where a token is wide: 64 to 1024
    if op == "rope":
        tokens = _log(rng, 1, 64 * room)
        seqs = _log(rng, 1, min(64, tokens))
        return dict(op=op, cache=rng.choice(["none", "e4m3", "bf16"]), type=kind, seqs=seqs, tokens=tokens,
                    ctx=tokens + _log(rng, 1, 100000), heads=kv_heads * rng.choice([1, 2, 4]),
                    kv_heads=kv_heads, dim=dim, rotary=rng.choice([dim // 4, dim // 2, dim]),
                    interleaved=rng.random() < 0.25, page=page)
    if op in ("write", "read"):
        tokens = _log(rng, 1, 256 * room)
        seqs = _log(rng, 1, min(64, tokens))
        return dict(op=op, cache=cache, type=kind, seqs=seqs, tokens=tokens,
                    ctx=tokens + _log(rng, 1, 4096), kv_heads=kv_heads, dim=dim, page=page)
    nodes = _log(rng, 1, 64)
    if op == "accept":
        return dict(op=op, cache=cache, seqs=_log(rng, 1, 256), nodes=nodes, ctx=nodes + _log(rng, 1, 1024),
                    kv_heads=kv_heads, dim=dim, page=page)
    groups = rng.choice([1, 2, 4, 8])
    seqs = _log(rng, 1, 64)
    # cached tokens x heads x width, and with them the rows, bounded below attend_large's
    most = 8 * 32768 * 8 * 128 // (seqs * kv_heads * dim)
    most = min(32768, most, most * 256 // (groups * nodes))
    return dict(op=op, cache=cache, seqs=seqs, nodes=nodes, ctx=_log(rng, nodes, max(nodes + 1, most)),
                ragged=rng.random() < 0.5, heads=kv_heads * groups, kv_heads=kv_heads, dim=dim, page=page,
                gate=rng.random() < 0.5)


def _spread(n, lo, hi):
    """n whole numbers in [lo, hi], spread unevenly, the same ones for a case at every seed."""
    return [lo + int((hi - lo) * ((0.6180339887 * (i + 1)) % 1.0)) for i in range(n)]


def _plan(case):
    """(tokens of each sequence, cached length of each sequence) of a case."""
    n, op = case["seqs"], case["op"]
    if op in ("rope", "write", "read"):
        share = [1 + x for x in _spread(n, 0, 1000)]
        left = case["tokens"] - n
        counts = [1 + left * s // sum(share) for s in share]
        counts[0] += case["tokens"] - sum(counts)
        lens = [min(max(c, case["ctx"] - i), case["ctx"]) for i, c in enumerate(counts)]
        if op == "read":
            lens = list(counts)
        return counts, [max(c, l) for c, l in zip(counts, lens)]
    if op == "accept":
        return [case["nodes"]] * n, [case["ctx"]] * n
    if not case["ragged"]:
        return [case["nodes"]] * n, [case["ctx"]] * n
    counts = [max(1, x) for x in _spread(n, case["nodes"] // 4, case["nodes"])]
    counts[0] = case["nodes"]
    lens = [max(c, x) for c, x in zip(counts, reversed(_spread(n, case["ctx"] // 8, case["ctx"])))]
    lens[-1] = max(lens[-1], case["ctx"])
    return counts, lens


def work(case):
    counts, lens = _plan(case)
    T, D, Hk = sum(counts), case["dim"], case["kv_heads"]
    elem = {"bf16": 2, "f32": 4}.get(case.get("type"), 2)
    held = {"e4m3": D + 4, "bf16": 2 * D, "none": 0}[case["cache"]]  # one cached row of one head
    if case["op"] == "rope":
        H = case["heads"]
        if case["cache"] == "none":
            b = 2 * T * (H + Hk) * D * elem
        else:
            b = T * ((2 * H + 2 * Hk) * D * elem + 2 * Hk * held)
        return {"bytes": b + 4 * T, "flops": 8 * T * (H + Hk) * D}
    if case["op"] in ("write", "read"):
        return {"bytes": 2 * T * Hk * (D * elem + held), "flops": 2 * T * Hk * D}
    if case["op"] == "accept":
        moved = case["seqs"] * (_depth(case["nodes"]) - 1)
        return {"bytes": 2 * 2 * moved * Hk * held + 4 * case["seqs"] * _depth(case["nodes"]), "flops": 0}
    H = case["heads"]
    b = 2 * sum(lens) * Hk * held + (3 if case["gate"] else 2) * T * H * D * 2
    return {"bytes": b, "flops": sum(4 * c * l * H * D for c, l in zip(counts, lens))}


# ---------------------------------------------------------------- the inputs

def _depth(nodes):
    """Nodes of the accepted path in a draft of that many."""
    return max(1, min(nodes, int(math.log2(nodes + 1)) + 1))


def _cache(gen, case, pages, filled):
    """A page pool; `filled`: holding quantised normal values, else zeros."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    made = {}
    for name in ("k", "v"):
        if case["cache"] == "bf16":
            x = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
            if filled:
                x.normal_(generator=gen)
            made[name], made[name + "_scale"] = x, None
            continue
        codes = torch.zeros(shape, dtype=torch.float8_e4m3fn, device=DEV)
        scale = torch.zeros(shape[:3], dtype=torch.float32, device=DEV)
        if filled:
            step = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
            for a in range(0, pages, step):
                x = torch.randn((min(step, pages - a),) + shape[1:], generator=gen, device=DEV)
                s = x.abs().amax(-1) / E4M3_MAX
                scale[a:a + step] = s
                codes[a:a + step] = (x / s[..., None]).to(torch.float8_e4m3fn)
        made[name], made[name + "_scale"] = codes, scale
    return made


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    counts, lens = _plan(case)
    n, T, ps, D, Hk = len(counts), sum(counts), case["page"], case["dim"], case["kv_heads"]
    i32 = dict(dtype=torch.int32, device=DEV)
    state = {"case": dict(case), "tokens": T, "max_nodes": max(counts)}
    state["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), **i32)
    state["lens"] = torch.tensor(lens, **i32)
    # pages in no order; only the pages that the call touches are there for calls that look at the
    # last tokens alone (an entry of -1: no page)
    last_only = case["op"] in ("rope", "write")
    first = [(l - c) // ps if last_only else 0 for c, l in zip(counts, lens)]
    need = [-(-l // ps) - f for f, l in zip(first, lens)]
    ids = rng.permutation(sum(need) + 2)
    table = np.full((n, max(-(-l // ps) for l in lens)), -1, np.int32)
    at = 0
    for i in range(n):
        table[i, first[i]:first[i] + need[i]] = ids[at:at + need[i]]
        at += need[i]
    state["table"] = torch.from_numpy(table).to(DEV)
    if case["cache"] != "none":
        state["cache"] = _cache(gen, case, len(ids), not last_only)
    kind = TYPES.get(case.get("type"), torch.bfloat16)
    if case["op"] == "rope":
        # the fused projection's output: q, k, v side by side in one row per token
        H = case["heads"]
        x = torch.randn((T, (H + 2 * Hk) * D), generator=gen, device=DEV).to(kind)
        state["q"], state["k"], state["v"] = (
            x[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, H), (H, H + Hk), (H + Hk, H + 2 * Hk)))
        state["q_w"], state["k_w"] = (1 + 0.1 * torch.randn(D, generator=gen, device=DEV) for _ in range(2))
        start = [l - c for c, l in zip(counts, lens)]
        state["pos"] = torch.tensor(np.concatenate([np.arange(s, s + c) for s, c in zip(start, counts)]), **i32)
        r = case["rotary"]
        state["inv_freq"] = 1e7 ** (-torch.arange(0, r, 2, dtype=torch.float64, device=DEV) / r)
    elif case["op"] == "write":
        state["k"], state["v"] = (torch.randn((T, Hk, D), generator=gen, device=DEV).to(kind) for _ in range(2))
    elif case["op"] == "accept":
        deep = _depth(case["nodes"])
        path = np.stack([np.concatenate([[0], 1 + np.sort(rng.permutation(case["nodes"] - 1)[:deep - 1])])
                         for _ in range(n)])
        state["path"] = torch.tensor(np.concatenate([path, np.full((n, 2), -1)], 1), **i32)
    elif case["op"] == "attend":
        H = case["heads"]
        state["q"] = torch.randn((T, H, D), generator=gen, device=DEV).to(torch.bfloat16)
        if case["gate"]:
            state["gate"] = torch.randn((T, H, D), generator=gen, device=DEV).to(torch.bfloat16)
        bits = []
        for c in counts:  # each node hangs on one of the nodes before it: a random tree
            seen = []
            for i in range(c):
                seen.append((1 << i) | (seen[int(rng.integers(max(0, i - 8), i))] if i else 0))
            bits += seen
        state["mask"] = torch.from_numpy(np.array(bits, np.uint64).view(np.int64)).to(DEV)
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _framework(state, case)
    return {"rope": _rope, "write": _write, "read": _read, "accept": _accept, "attend": _attend}[case["op"]](
        state, case)


def _framework(s, case):
    import gated_deltanet_linear_silu_b200 as gdn

    where = (s["table"], s["lens"], s["cu"])
    kv = gdn.KVCache(**s["cache"]) if "cache" in s else None
    if case["op"] == "rope":
        if case["cache"] == "none":
            q, k = gdn.qk_norm_rope(s["q"], s["k"], s["q_w"], s["k_w"], s["pos"], s["inv_freq"],
                                    interleaved=case["interleaved"])
            return {"q": q, "k": k}
        q = gdn.qk_norm_rope_cache(s["q"], s["k"], s["v"], s["q_w"], s["k_w"], s["pos"], s["inv_freq"], kv,
                                   *where, interleaved=case["interleaved"])
        return {"q": q, **_held(s)}
    if case["op"] == "write":
        gdn.kv_cache_write(s["k"], s["v"], kv, *where)
        return _held(s)
    if case["op"] == "read":
        k, v = gdn.kv_cache_read(kv, *where, n_tokens=s["tokens"], dtype=TYPES[case["type"]])
        return {"k": k, "v": v}
    if case["op"] == "accept":
        return {"lens": gdn.kv_cache_accept(kv, *where, s["path"]), **_held(s)}
    o, lse = gdn.tree_attention(s["q"], kv, *where, mask=s["mask"], max_nodes=s["max_nodes"],
                                gate=s.get("gate"), return_lse=True)
    return {"o": o, "lse": lse}


def _held(s):
    """The cache's contents: e4m3 values with their scales, or bf16 values."""
    return {name: x for name, x in s["cache"].items() if x is not None}


def _places(s, case):
    """(page, row in it) of each packed token."""
    cu, T = s["cu"].long(), s["tokens"]
    t = torch.arange(T, device=DEV)
    n = torch.searchsorted(cu, t, right=True) - 1
    at = s["lens"].long()[n] - cu[n + 1] + t
    return s["table"].long()[n, at // case["page"]], at % case["page"]


def _put(s, case, name, x, page, row):
    """Stores the rows x [T, Hk, D] (fp32) in the cache, quantised where it is."""
    if s["cache"][name + "_scale"] is None:
        s["cache"][name][page, :, row] = x.to(torch.bfloat16)
        return
    scale = x.abs().amax(-1) / E4M3_MAX
    code = (x / scale[..., None]).to(torch.float8_e4m3fn)
    s["cache"][name].view(torch.uint8)[page, :, row] = code.view(torch.uint8)
    s["cache"][name + "_scale"][page, :, row] = scale


def _rotate(x, cos, sin, r, interleaved):
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., r:]], -1)


def _rope(s, case):
    angle = s["pos"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    got = {}
    for name in ("q", "k"):
        x = s[name].float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s[name + "_w"]
        got[name] = _rotate(x, cos, sin, case["rotary"], case["interleaved"])
    if case["cache"] == "none":
        return {name: x.to(s["q"].dtype) for name, x in got.items()}
    page, row = _places(s, case)
    _put(s, case, "k", got["k"], page, row)
    _put(s, case, "v", s["v"].float(), page, row)
    return {"q": got["q"].to(s["q"].dtype), **_held(s)}


def _write(s, case):
    page, row = _places(s, case)
    _put(s, case, "k", s["k"].float(), page, row)
    _put(s, case, "v", s["v"].float(), page, row)
    return _held(s)


def _rows(s, name, page, row):
    x = s["cache"][name]
    if s["cache"][name + "_scale"] is None:
        return x[page, :, row].float()
    codes = x.view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn)
    return codes.float() * s["cache"][name + "_scale"][page, :, row][..., None]


def _read(s, case):
    page, row = _places(s, case)
    return {name: _rows(s, name, page, row).to(TYPES[case["type"]]) for name in ("k", "v")}


def _accept(s, case):
    cu, path, ps = s["cu"].long(), s["path"].long(), case["page"]
    base = (s["lens"].long() - (cu[1:] - cu[:-1]))[:, None]
    kept = path >= 0
    table = s["table"].long()
    n = torch.arange(path.shape[0], device=DEV)[:, None].expand_as(path)[kept]
    source = (base + path)[kept]
    target = (base + torch.arange(path.shape[1], device=DEV))[kept]
    for x in _held(s).values():
        x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
        x[table[n, target // ps], :, target % ps] = x[table[n, source // ps], :, source % ps]
    return {"lens": (base[:, 0] + kept.sum(1)).to(torch.int32), **_held(s)}


def _attend(s, case):
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    cu, lens, T = s["cu"].long(), s["lens"].long(), s["tokens"]
    N, most, longest = lens.numel(), s["max_nodes"], s["table"].shape[1] * case["page"]
    # every sequence's keys and values, dense: [N, Hk, longest, D]
    table = s["table"].long().clamp(min=0)
    dense = {}
    for name in ("k", "v"):
        x = s["cache"][name]
        if s["cache"][name + "_scale"] is None:
            x = x[table].float()
        else:
            x = x.view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * s["cache"][name + "_scale"][table][..., None]
        dense[name] = x.transpose(1, 2).reshape(N, Hk, longest, D)
    # queries padded to the most nodes: [N, Hk, most * H / Hk, D]
    t = torch.arange(T, device=DEV)
    n = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[n]
    q = torch.zeros((N, most, H, D), device=DEV)
    q[n, i] = s["q"].float()
    q = q.view(N, most, Hk, H // Hk, D).transpose(1, 2).reshape(N, Hk, -1, D)
    score = (q @ dense["k"].transpose(2, 3)).view(N, Hk, most, H // Hk, longest) * D ** -0.5
    # a node sees the context before the draft and the drafted nodes whose bit it has
    bits = torch.zeros((N, most), dtype=torch.int64, device=DEV)
    bits[n, i] = s["mask"]
    pos = torch.arange(longest, device=DEV)
    base = (lens - (cu[1:] - cu[:-1]))[:, None]
    drafted = (pos - base).clamp(0, 63)
    sees = (pos < base)[:, None] | ((pos >= base) & (pos < lens[:, None]))[:, None] & (
        (bits[:, :, None] >> drafted[:, None]) & 1).bool()
    score = score.masked_fill(~sees[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ dense["v"]).view(N, Hk, most, H // Hk, D) / total.clamp(min=1e-30)
    lse = (top + total.log())[..., 0]
    o = o.transpose(1, 2).reshape(N, most, H, D)[n, i]
    lse = lse.transpose(1, 2).reshape(N, most, H)[n, i]
    if case["gate"]:
        o = o * torch.sigmoid(s["gate"].float())
    return {"o": o.to(s["q"].dtype), "lse": lse}


# ---------------------------------------------------------------- from the definition, in 64 bits

def _e4m3(x):
    """The e4m3 values nearest to x, ties to even: steps of 2^(e-3), at least 2^-9, up to 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    e = torch.where(x.abs() >= 2.0 ** (e + 1), e + 1, e)
    step = 2.0 ** (e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _each(s):
    """(sequence, its tokens' slice, its cached length, its page ids) of every sequence."""
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].cpu().numpy()
    return [(n, slice(cu[n], cu[n + 1]), lens[n], table[n]) for n in range(len(lens))]


def _spots(ids, at, ps):
    at = np.asarray(at)
    return (torch.from_numpy(ids[at // ps].astype(np.int64)).to(DEV), torch.from_numpy(at % ps).to(DEV))


def exact(case, seed):
    s = prepare(case, seed)
    ps, op = case["page"], case["op"]
    out = {name: x.double() for name, x in _held(s).items()} if case["cache"] != "none" else {}
    scaled = case["cache"] == "e4m3"

    def turned(name):
        x, w, r = s[name].double(), s[name + "_w"].double(), case["rotary"]
        x = x / (x.pow(2).sum(-1, keepdim=True) / case["dim"] + 1e-6).sqrt() * w
        a = (s["pos"].double()[:, None] * s["inv_freq"])[:, None]
        z = torch.view_as_complex((x[..., :r].unflatten(-1, (r // 2, 2)) if case["interleaved"] else
                                   x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)).contiguous())
        z = torch.view_as_real(z * torch.polar(torch.ones_like(a), a))
        z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, x[..., r:]], -1)

    def store(name, x):
        for n, span, length, ids in _each(s):
            m = span.stop - span.start
            page, row = _spots(ids, np.arange(length - m, length), ps)
            y = x[span]
            if scaled:
                scale = y.abs().amax(-1) / E4M3_MAX
                out[name + "_scale"][page, :, row] = scale
                y = _e4m3(y / scale[..., None])
            out[name][page, :, row] = y

    def values(name, page, row):
        x = out[name][page, :, row]
        return x * out[name + "_scale"][page, :, row][..., None] if scaled else x

    if op == "rope":
        q, k = turned("q"), turned("k")
        if case["cache"] == "none":
            return {"q": q, "k": k}
        store("k", k)
        store("v", s["v"].double())
        return {"q": q, **out}
    if op == "write":
        store("k", s["k"].double())
        store("v", s["v"].double())
        return out
    if op == "read":
        got = {"k": [], "v": []}
        for n, span, length, ids in _each(s):
            m = span.stop - span.start
            for name in got:
                got[name].append(values(name, *_spots(ids, np.arange(length - m, length), ps)))
        return {name: torch.cat(x) for name, x in got.items()}
    if op == "accept":
        for n, span, length, ids in _each(s):
            path = [p for p in s["path"][n].tolist() if p >= 0]
            base = length - (span.stop - span.start)
            before = {name: x[_spots(ids, np.array(path) + base, ps)[0], :, _spots(ids, np.array(path) + base, ps)[1]].clone()
                      for name, x in out.items()}
            page, row = _spots(ids, np.arange(base, base + len(path)), ps)
            for name, x in out.items():
                x[page, :, row] = before[name]
        return {"lens": None, **out}
    H, Hk = case["heads"], case["kv_heads"]
    o, lse = [], []
    pools, out = out, {}
    for n, span, length, ids in _each(s):
        m = span.stop - span.start
        out = pools
        page, row = _spots(ids, np.arange(length), ps)
        k, v = (values(name, page, row).repeat_interleave(H // Hk, 1) for name in ("k", "v"))
        score = torch.einsum("ihd,jhd->hij", s["q"][span].double(), k) / math.sqrt(case["dim"])
        seen = torch.ones((m, length), dtype=torch.bool)
        for i, word in enumerate(s["mask"][span].tolist()):
            seen[i, length - m:] = torch.tensor([bool(word >> j & 1) for j in range(m)])
        score = torch.where(seen.to(DEV)[None], score, -math.inf)
        z = torch.logsumexp(score, -1)
        o.append(torch.einsum("hij,jhd->ihd", torch.exp(score - z[..., None]), v))
        lse.append(z.T)
    o = torch.cat(o)
    if case["gate"]:
        o = o / (1 + torch.exp(-s["gate"].double()))
    return {"o": o, "lse": torch.cat(lse)}
