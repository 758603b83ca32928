"""The serving operators beside the linear layer, as cases to be timed: rotary
positions, the append of keys and values to a paged cache, and attention of
new tokens over that cache.

Shapes are those of decoder blocks like the benchmark's (32 query heads, 8 key
and value heads of 128: its q, k and v projections) and of generic others.
`run` computes a case in elementary torch operations in 32 bits, or, where
`own` is true, by the library's calls.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
MAX_POS = 131072


def listed():
    return [
        # one image's patches in a vision tower: two axes (height, width), 16 heads of 80
        dict(name="rope_image", op="rope", tokens=1161, heads=32, dim=80, rot=80, axes=2, pairs="interleaved", dtype="f16"),
        # the queries and keys of a long video prompt, three axes (time, height, width), out of a fused projection
        dict(name="rope_video", op="rope", tokens=16384, heads=40, dim=128, rot=128, axes=3, pairs="halves", dtype="bf16"),
        # one sequence decoding: the call is all latency
        dict(name="append_one", op="append", tokens=1, q_heads=32, kv_heads=8, dim=128, rot=128, axes=1, pairs="halves",
             dtype="bf16", cache="bf16", page=16, layout="heads"),
        # a decode batch into a cache of e4m3 codes
        dict(name="append_decode_e4m3", op="append", tokens=97, q_heads=32, kv_heads=8, dim=128, rot=128, axes=1,
             pairs="halves", dtype="bf16", cache="e4m3", page=64, layout="heads"),
        # a long prompt, rotation of half of each head, cache laid out token by token
        dict(name="append_prompt", op="append", tokens=8192, q_heads=32, kv_heads=8, dim=128, rot=64, axes=1,
             pairs="halves", dtype="bf16", cache="bf16", page=16, layout="tokens"),
        # one sequence decoding at a short length: latency
        dict(name="attend_one", op="attend", seqs=1, kv_heads=8, group=4, dim=128, page=16, dtype="bf16", cache="bf16",
             layout="heads", new_lo=1, new_hi=1, len_lo=1009, len_hi=1009, window=0, empty=0, mix=1),
        # a decode batch of ragged lengths: the cache's bytes
        dict(name="attend_decode", op="attend", seqs=96, kv_heads=8, group=4, dim=128, page=16, dtype="bf16",
             cache="bf16", layout="heads", new_lo=1, new_hi=1, len_lo=300, len_hi=12000, window=0, empty=0, mix=2),
        # two very long sequences on a cache of e4m3 codes
        dict(name="attend_long_e4m3", op="attend", seqs=2, kv_heads=8, group=8, dim=128, page=64, dtype="bf16",
             cache="e4m3", layout="heads", new_lo=1, new_hi=1, len_lo=90000, len_hi=131071, window=0, empty=0, mix=3),
        # a whole prompt: compute
        dict(name="attend_prompt", op="attend", seqs=1, kv_heads=8, group=4, dim=128, page=16, dtype="bf16",
             cache="bf16", layout="tokens", new_lo=8192, new_hi=8192, len_lo=8192, len_hi=8192, window=0, empty=0, mix=4),
        # chunks of prompts whose beginning is already in a cache of e4m3 codes
        dict(name="attend_chunks_e4m3", op="attend", seqs=3, kv_heads=8, group=4, dim=128, page=32, dtype="f16",
             cache="e4m3", layout="heads", new_lo=500, new_hi=1030, len_lo=9000, len_hi=16000, window=0, empty=0, mix=5),
        # prompts' chunks and decoding sequences in one batch, heads of 64 in groups of 7, a sliding window,
        # and padded entries that have no tokens in the cache
        dict(name="attend_mixed_window", op="attend", seqs=17, kv_heads=4, group=7, dim=64, page=32, dtype="f16",
             cache="f16", layout="tokens", new_lo=1, new_hi=600, len_lo=100, len_hi=5000, window=1024, empty=2, mix=6),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo .. hi."""
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dim = rng.choice([64, 80, 96, 128])
    dtype = rng.choice(["bf16", "f16"])
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
    layout = rng.choice(["heads", "tokens"])
    cache = rng.choice([dtype, "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    axes = rng.choice([1, 1, 2, 3])
    pairs = rng.choice(["halves", "interleaved"])
    rot = rng.choice([dim, dim, 64 if dim >= 64 else dim, 32])
    op = rng.choice(["rope", "append", "decode", "decode", "chunks", "chunks"])
    if op == "rope":
        return dict(op="rope", tokens=_log(rng, 5, 16000), heads=kv_heads * (group + 1), dim=dim, rot=rot, axes=axes,
                    pairs=pairs, dtype=dtype)
    if op == "append":
        return dict(op="append", tokens=_log(rng, 1, 8190), q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, rot=rot,
                    axes=axes, pairs=pairs, dtype=dtype, cache=cache, page=page, layout=layout)
    if op == "decode":
        hi = _log(rng, 200, 60000)
        seqs = _log(rng, 1, max(1, min(96, 500000 // hi)))
        return dict(op="attend", seqs=seqs, kv_heads=kv_heads, group=group, dim=dim, page=page, dtype=dtype, cache=cache,
                    layout=layout, new_lo=1, new_hi=rng.choice([1, 1, 4]), len_lo=_log(rng, 1, hi), len_hi=hi,
                    window=rng.choice([0, 0, 0, 700]), empty=0, mix=rng.randrange(10 ** 6))
    new = _log(rng, 16, 4000)
    hi = _log(rng, new, max(new, min(20000, 24000000 // new)))
    room = 8192 * 8192 * 32 // (new * hi * kv_heads * group)
    seqs = _log(rng, 1, max(1, min(24, room // 2)))
    return dict(op="attend", seqs=seqs, kv_heads=kv_heads, group=group, dim=dim, page=page, dtype=dtype, cache=cache,
                layout=layout, new_lo=_log(rng, 1, new), new_hi=new, len_lo=_log(rng, 1, hi), len_hi=hi,
                window=rng.choice([0, 0, 0, 500]), empty=0, mix=rng.randrange(10 ** 6))


def _sections(rot, axes):
    """Pairs of a head that turn by each axis' position: about equal shares."""
    half = rot // 2
    cut = [half * a // axes for a in range(axes + 1)]
    return [cut[a + 1] - cut[a] for a in range(axes)]


def _lengths(case):
    """(new tokens, tokens in the cache with them) of each sequence: the case's own, whatever the seed."""
    r = random.Random(case["mix"])
    new = [_log(r, case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    new[r.randrange(len(new))] = case["new_hi"]
    lens = [max(n, _log(r, case["len_lo"], case["len_hi"])) for n in new]
    lens[r.randrange(len(lens))] = case["len_hi"]
    lens = [max(n, t) for n, t in zip(new, lens)]
    for i in range(case["empty"]):
        new[i], lens[i] = 1, 0
    return new, lens


def _table(rot, device):
    """cos and sin of rot / 2 angles for each position."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    angle = torch.arange(MAX_POS, device=device, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _cache_pair(case, pages, gen, filled):
    """Key and value caches [pages, kv_heads, page, dim] in the case's memory order, with their scales."""
    dev, dim, heads, page = gen.device, case["dim"], case["kv_heads"], case["page"]
    order = (pages, heads, page, dim) if case["layout"] == "heads" else (pages, page, heads, dim)
    got = []
    for _ in range(2):
        if case["cache"] == "e4m3":
            codes, scales = torch.zeros(order, dtype=torch.uint8, device=dev), torch.ones((pages, heads, page), device=dev)
            t = codes if case["layout"] == "heads" else codes.transpose(1, 2)
            for at in range(0, pages if filled else 0, 512):
                x = torch.randn((min(512, pages - at), heads, page, dim), generator=gen, device=dev)
                s = x.abs().amax(-1) / 448.0
                scales[at:at + 512] = s
                t[at:at + 512] = (x / s[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
            got.append((t, scales))
        else:
            t = torch.zeros(order, dtype=DTYPES[case["cache"]], device=dev)
            if filled:
                t.normal_(generator=gen)
            got.append((t if case["layout"] == "heads" else t.transpose(1, 2), None))
    return got


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(int(seed) * 7919 + 13)
    s = dict(case=case)
    if case["op"] in ("rope", "append"):
        tokens, rot, axes = case["tokens"], case["rot"], case["axes"]
        s["table"] = _table(rot, dev)
        s["sections"] = _sections(rot, axes)
        s["axis"] = torch.repeat_interleave(torch.arange(axes, device=dev), torch.tensor(s["sections"], device=dev))
        s["positions"] = torch.randint(0, MAX_POS, (axes, tokens), generator=gen, device=dev, dtype=torch.int32)
    if case["op"] == "rope":
        # queries and keys as the leading columns of a wider row, as a fused projection leaves them
        row = torch.empty((tokens, case["heads"] + 8, case["dim"]), device=dev, dtype=DTYPES[case["dtype"]])
        s["x"] = row.normal_(generator=gen)[:, :case["heads"]]
    elif case["op"] == "append":
        heads, kv = case["q_heads"], case["kv_heads"]
        row = torch.empty((tokens, heads + 2 * kv, case["dim"]), device=dev, dtype=DTYPES[case["dtype"]])
        row.normal_(generator=gen)
        s["q"], s["k"], s["v"] = row[:, :heads], row[:, heads:heads + kv], row[:, heads + kv:]
        pages = tokens // case["page"] + 9
        s["slots"] = torch.randperm(pages * case["page"], generator=gen, device=dev)[:tokens]
        if tokens > 256:  # a prompt fills whole pages in order, the pages being anywhere
            where = torch.randperm(pages, generator=gen, device=dev)
            at = torch.arange(tokens, device=dev)
            s["slots"] = where[at // case["page"]] * case["page"] + at % case["page"]
        (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _cache_pair(case, pages, gen, False)
    else:
        new, lens = _lengths(case)
        page, heads = case["page"], case["kv_heads"] * case["group"]
        need = [-(-t // page) for t in lens]
        pages = sum(need) + 5
        where = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        wide = max(need) + 1
        col = torch.arange(wide, device=dev)
        first = torch.tensor([0] + need, device=dev).cumsum(0)[:-1]
        used = col[None, :] < torch.tensor(need, device=dev)[:, None]
        s["block_table"] = torch.where(used, where[(first[:, None] + col[None, :]).clamp(max=pages - 1)], 0).to(torch.int32).contiguous()
        s["lens"] = torch.tensor(lens, device=dev, dtype=torch.int32)
        s["starts"] = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
        s["new"], s["tokens"], s["max_new"], s["max_len"] = new, sum(new), max(new), max(lens)
        # queries as the leading columns of a fused projection's rows
        row = torch.empty((s["tokens"], heads + 2 * case["kv_heads"], case["dim"]), device=dev, dtype=DTYPES[case["dtype"]])
        s["q"] = row.normal_(generator=gen)[:, :heads]
        (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _cache_pair(case, pages, gen, True)
        # where each token's row stands in a rectangle of sequences, for the plain form
        s["seq_of"] = torch.repeat_interleave(torch.arange(len(new), device=dev), torch.tensor(new, device=dev))
        s["index_of"] = torch.arange(s["tokens"], device=dev) - s["starts"].long()[s["seq_of"]]
    if own:
        import fp8_weight_only_gb300 as fw
        s["fw"] = fw
        if case["op"] != "attend":
            s["rope"] = fw.Rope(s["table"], sections=s["sections"], interleaved=case["pairs"] == "interleaved")
        if case["op"] != "rope":
            s["cache"] = fw.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
    return s


def _turn(x, s):
    """x [tokens, heads, dim] in 32 bits, the first rot values of each head rotated."""
    case = s["case"]
    rot, x = case["rot"], x.float()
    half = rot // 2
    at = s["positions"].long()[s["axis"]].t()
    i = torch.arange(half, device=x.device)
    cos, sin = s["table"][at, i][:, None], s["table"][at, half + i][:, None]
    if case["pairs"] == "halves":
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _put(cache, scales, x, s):
    """Rows x [tokens, kv_heads, dim] in 32 bits into their slots."""
    page = s["case"]["page"]
    at, off = s["slots"] // page, s["slots"] % page
    if scales is None:
        cache[at, :, off] = x.to(cache.dtype)
    else:
        scale = x.abs().amax(-1) / 448.0
        scale = torch.where(scale == 0, torch.ones_like(scale), scale)
        cache[at, :, off] = (x / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[at, :, off] = scale


def _caches(s):
    """The cache after an append, codes as the values they stand for."""
    if s["ks"] is None:
        return dict(k=s["kc"], v=s["vc"])
    return dict(k=s["kc"].view(torch.float8_e4m3fn), v=s["vc"].view(torch.float8_e4m3fn), k_scales=s["ks"], v_scales=s["vs"])


def _gathered(cache, scales, table):
    """The cached rows of each sequence in order, [seqs, kv_heads, width * page, dim] in 32 bits."""
    t = cache[table.long()]
    t = t.float() if scales is None else t.view(torch.float8_e4m3fn).float() * scales[table.long()][..., None]
    return t.transpose(1, 2).flatten(2, 3)


def _attend(s):
    case = s["case"]
    heads, group, dim = case["kv_heads"], case["group"], case["dim"]
    seqs, most = case["seqs"], s["max_new"]
    k = _gathered(s["kc"], s["ks"], s["block_table"])
    q = torch.zeros((seqs, most, heads, group, dim), device=k.device)
    q[s["seq_of"], s["index_of"]] = s["q"].float().view(-1, heads, group, dim)
    q = q.permute(0, 2, 1, 3, 4).reshape(seqs, heads, most * group, dim)
    scores = (q @ k.transpose(2, 3)).view(seqs, heads, most, group, -1) * (1.0 / math.sqrt(dim))
    del k
    new = s["starts"][1:] - s["starts"][:-1]
    last = (s["lens"] - new)[:, None] + torch.arange(most, device=q.device)
    at = torch.arange(scores.shape[-1], device=q.device)
    seen = at <= last[..., None]
    if case["window"]:
        seen &= at > (last - case["window"])[..., None]
    scores.masked_fill_(~seen[:, None, :, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    weight = scores.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    total = weight.sum(-1, keepdim=True)
    v = _gathered(s["vc"], s["vs"], s["block_table"])
    out = weight.view(seqs, heads, most * group, -1) @ v
    out = out.view(seqs, heads, most, group, dim) / torch.where(total == 0, torch.ones_like(total), total)
    out = out.permute(0, 2, 1, 3, 4).reshape(seqs, most, heads * group, dim)
    return out[s["seq_of"], s["index_of"]].to(s["q"].dtype)


def run(s):
    case = s["case"]
    if own:
        fw = s["fw"]
        if case["op"] == "rope":
            return fw.rope(s["x"], s["positions"], s["rope"])
        if case["op"] == "append":
            return dict(q=fw.rope_append(s["q"], s["k"], s["v"], s["slots"], s["cache"], s["positions"], s["rope"]), **_caches(s))
        return fw.paged_attention(s["q"], s["cache"], s["block_table"], s["lens"],
                                  starts=s["starts"] if case["new_hi"] > 1 else None, window=case["window"],
                                  max_new=s["max_new"], max_len=s["max_len"])
    if case["op"] == "rope":
        return _turn(s["x"], s).to(s["x"].dtype)
    if case["op"] == "append":
        _put(s["kc"], s["ks"], _turn(s["k"], s), s)
        _put(s["vc"], s["vs"], s["v"].float(), s)
        return dict(q=_turn(s["q"], s).to(s["q"].dtype), **_caches(s))
    return _attend(s)


def _pairs(case):
    """Query and key pairs that are seen, and cached tokens that any row of their sequence sees, over all sequences."""
    seen = read = 0
    for n, t in zip(*_lengths(case)):
        if not t:
            continue
        w = case["window"] or t
        full = [min(w, t - n + 1), min(w, t)]
        ramp = full[1] - full[0]  # rows whose count still grows by one
        seen += (full[0] + full[1]) * (ramp + 1) // 2 + (n - ramp - 1) * full[1]
        read += min(t, w + n - 1)
    return seen, read


def work(case):
    if case["op"] == "rope":
        row = case["tokens"] * case["heads"] * case["dim"]
        rows = min(MAX_POS, case["tokens"] * case["axes"])
        return {"bytes": 4 * row + 4 * case["axes"] * case["tokens"] + 4 * rows * case["rot"] // case["axes"],
                "flops": 3 * row * case["rot"] // case["dim"]}
    if case["op"] == "append":
        q, kv = case["tokens"] * case["q_heads"] * case["dim"], case["tokens"] * case["kv_heads"] * case["dim"]
        held = 2 * kv + 8 * case["tokens"] * case["kv_heads"] if case["cache"] == "e4m3" else 4 * kv
        rows = min(MAX_POS, case["tokens"] * case["axes"])
        return {"bytes": 4 * q + 4 * kv + held + (4 * case["axes"] + 8) * case["tokens"] + 4 * rows * case["rot"] // case["axes"],
                "flops": 3 * (q + kv) * case["rot"] // case["dim"]}
    seen, read = _pairs(case)
    heads, dim = case["kv_heads"] * case["group"], case["dim"]
    each = 2 * dim + 8 if case["cache"] == "e4m3" else 4 * dim
    return {"bytes": read * case["kv_heads"] * each + 4 * sum(_lengths(case)[0]) * heads * dim, "flops": 4 * seen * heads * dim}


def exact(case, seed):
    """The case's outputs in 64 bits from the definition: complex turns, and one softmax for each sequence and head."""
    s = prepare(case, seed)

    def turned(x):
        rot = case["rot"]
        half, x = rot // 2, x.double().clone()
        at = torch.stack([s["positions"][a].long() for a in s["axis"].tolist()], 1)
        rows = s["table"].double()
        unit = torch.complex(rows[:, :half].gather(0, at), rows[:, half:].gather(0, at))[:, None]
        if case["pairs"] == "halves":
            z = torch.complex(x[..., :half], x[..., half:rot]) * unit
            x[..., :half], x[..., half:rot] = z.real, z.imag
        else:
            z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * unit
            x[..., 0:rot:2], x[..., 1:rot:2] = z.real, z.imag
        return x

    if case["op"] == "rope":
        return turned(s["x"])
    if case["op"] == "append":
        got = dict(q=turned(s["q"]))
        for name, x in (("k", turned(s["k"])), ("v", s["v"].double())):
            page, off = torch.div(s["slots"], case["page"], rounding_mode="floor"), s["slots"].remainder(case["page"])
            if case["cache"] == "e4m3":
                scales = s[name + "s"].double()
                top = x.abs().max(-1).values
                scales[page, :, off] = torch.where(top > 0, top / 448, torch.ones_like(top))
                got[name], got[name + "_scales"] = None, scales
            else:
                held = s[name + "c"].double()
                held[page, :, off] = x
                got[name] = held
        return got
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lens, table, starts = s["lens"].tolist(), s["block_table"].long(), s["starts"].tolist()
    for b, n in enumerate(s["new"]):
        t = lens[b]
        if not t:
            continue
        pages = table[b, :-(-t // case["page"])]
        rows = torch.arange(t - n, t, device=out.device)[:, None]
        cols = torch.arange(t, device=out.device)[None, :]
        hidden = cols > rows
        if case["window"]:
            hidden |= rows - cols >= case["window"]
        for h in range(case["kv_heads"]):
            kv = []
            for c, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
                x = c[pages, h].flatten(0, 1)[:t]
                x = x.double() if sc is None else x.view(torch.float8_e4m3fn).double() * sc[pages, h].flatten()[:t, None].double()
                kv.append(x)
            for g in range(h * case["group"], (h + 1) * case["group"]):
                q = s["q"][starts[b]:starts[b + 1], g].double()
                z = (q @ kv[0].t()) / math.sqrt(case["dim"])
                out[starts[b]:starts[b + 1], g] = torch.softmax(z.masked_fill_(hidden, float("-inf")), -1) @ kv[1]
    return out
