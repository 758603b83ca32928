"""The 4-bit forms of the layer, as cases to be timed: weights in 4 bits (their
quantisation, and the linear layer on them) and a paged cache of keys and values
in 4 bits (the append to it, and attention over it).

One form serves both.  A row of values (an output channel's weights, a slot and
head of the cache) has 4-bit e2m1 codes, two a byte with the first in the low
half, an e4m3 byte for each 16 of them, and one 32-bit scale:
    value = scale * e4m3(block) * e2m1(code).

Shapes are those of decoder blocks like the benchmark's (hidden size 4096, 14336
in the middle, 32 query heads, 8 key and value heads of 128) and generic others.
`run` computes a case in elementary torch operations in 32 bits, or, where `own`
is true, by the library's calls.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
MAX_POS = 131072


def listed():
    return [
        # a key projection for one token: the call is all latency
        dict(name="linear_one_small", op="linear", m=1, n=1024, k=4096, dtype="bf16", bias=False),
        # the projection back from the middle for one token: the weight's bytes
        dict(name="linear_one_down", op="linear", m=1, n=4096, k=14336, dtype="bf16", bias=False),
        # a small batch decoding, with a bias, sizes that divide nothing
        dict(name="linear_batch_odd", op="linear", m=23, n=10007, k=4128, dtype="f16", bias=True),
        # a prompt: compute
        dict(name="linear_prompt", op="linear", m=2048, n=14336, k=4096, dtype="bf16", bias=False),
        # a small matrix quantised and read back (its error looked at, say)
        dict(name="requantize_small", op="requantize", n=1001, k=992, dtype="bf16", out="f32"),
        # a large one, from the 32-bit weights of a checkpoint
        dict(name="requantize_large", op="requantize", n=14336, k=4096, dtype="f32", out="bf16"),
        # one token decoding into the cache
        dict(name="append_one", op="append", tokens=1, q_heads=32, kv_heads=8, dim=128, rot=128, axes=1, pairs="halves",
             dtype="bf16", page=16),
        # a long prompt, rotation of half of each head
        dict(name="append_prompt", op="append", tokens=8192, q_heads=32, kv_heads=8, dim=128, rot=64, axes=1,
             pairs="interleaved", dtype="f16", page=64),
        # one sequence decoding at a short length: latency
        dict(name="attend_one", op="attend", seqs=1, kv_heads=8, group=4, dim=128, page=16, dtype="bf16", layout="heads",
             new_lo=1, new_hi=1, len_lo=1009, len_hi=1009, window=0, empty=0, mix=1),
        # a decode batch of ragged lengths, padded entries without tokens among them: the cache's bytes
        dict(name="attend_decode", op="attend", seqs=96, kv_heads=8, group=4, dim=128, page=16, dtype="bf16",
             layout="heads", new_lo=1, new_hi=1, len_lo=300, len_hi=12000, window=0, empty=2, mix=2),
        # two very long sequences
        dict(name="attend_long", op="attend", seqs=2, kv_heads=8, group=8, dim=128, page=64, dtype="f16", layout="tokens",
             new_lo=1, new_hi=1, len_lo=90000, len_hi=131071, window=0, empty=0, mix=3),
        # chunks of prompts whose beginning is in the cache
        dict(name="attend_chunks", op="attend", seqs=3, kv_heads=8, group=4, dim=128, page=32, dtype="bf16",
             layout="heads", new_lo=500, new_hi=1030, len_lo=9000, len_hi=16000, window=0, empty=0, mix=5),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo .. hi."""
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "f16"])
    op = rng.choice(["linear", "linear", "linear", "requantize", "append", "decode", "decode", "chunks"])
    if op == "linear":
        n, k = _log(rng, 60, 16000), 32 * _log(rng, 2, 500)
        most = max(1, min(2040, 2048 * 14336 * 4096 // (n * k)))
        m = rng.choice([1, 1, _log(rng, 2, 64), _log(rng, 2, 64), _log(rng, 1, most)])
        return dict(op="linear", m=min(m, most), n=n, k=k, dtype=dtype, bias=rng.random() < 0.5)
    if op == "requantize":
        n = _log(rng, 20, 16000)
        k = 32 * _log(rng, 1, min(1000, 14336 * 4096 // (32 * n)))
        return dict(op=op, n=n, k=k, dtype=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["f32", "bf16", "f16"]))
    dim, page = rng.choice([32, 64, 96, 128, 128]), rng.choice([16, 32, 64, 128])
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 8190), q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim, 32, dim // 2]), axes=rng.choice([1, 1, 2, 3]),
                    pairs=rng.choice(["halves", "interleaved"]), dtype=dtype, page=page)
    layout = rng.choice(["heads", "tokens"])
    if op == "decode":
        hi = _log(rng, 200, 60000)
        seqs = _log(rng, 1, max(1, min(96, 500000 // hi)))
        return dict(op="attend", seqs=seqs, kv_heads=kv_heads, group=group, dim=dim, page=page, dtype=dtype,
                    layout=layout, new_lo=1, new_hi=rng.choice([1, 1, 4]), len_lo=_log(rng, 1, hi), len_hi=hi,
                    window=rng.choice([0, 0, 0, 700]), empty=0, mix=rng.randrange(10 ** 6))
    new = _log(rng, 16, 1030)
    hi = _log(rng, new, 16000)
    room = 3 * 1030 * 16000 * 32 // (new * hi * kv_heads * group)
    seqs = _log(rng, 1, max(1, min(24, room // 2)))
    return dict(op="attend", seqs=seqs, kv_heads=kv_heads, group=group, dim=dim, page=page, dtype=dtype, layout=layout,
                new_lo=_log(rng, 1, new), new_hi=new, len_lo=_log(rng, 1, hi), len_hi=hi,
                window=rng.choice([0, 0, 0, 500]), empty=0, mix=rng.randrange(10 ** 6))


# ------------------------------------------------------------------ the form --

def _quantized(x):
    """Rows x [..., k] in 32 bits -> (codes [..., k] in 0..15, blocks [..., k / 16] float8, scales [...])."""
    amax = x.abs().amax(-1)
    scales = torch.where(amax == 0, torch.ones_like(amax), (amax * (1.0 / 2688.0)).clamp_min(2.0 ** -126))
    y = x * (1.0 / scales)[..., None]
    blocks = (y.abs().unflatten(-1, (-1, 16)).amax(-1) * (1.0 / 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    b = blocks.float()
    inverse = torch.where(b == 0, torch.zeros_like(b), 1.0 / b)
    y = y * inverse.repeat_interleave(16, -1)
    a = y.abs()
    # to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; from the middle of two to the even code
    code = (a > 0.25).to(torch.uint8)
    for edge, takes in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= edge) if takes else (a > edge)
    return code + 8 * torch.signbit(y).to(torch.uint8), blocks, scales


def _packed(codes):
    """Two codes a byte, the first in the low half."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _values(codes, blocks, scales):
    """Packed codes [..., k / 2], bytes of blocks [..., k / 16], scales [...] -> the values in 32 bits."""
    half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([half, -half])
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    b = blocks.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)
    return v * b * scales[..., None]


# -------------------------------------------------------------------- inputs --

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


def _cache_half(case, pages, gen, filled, layout):
    """Keys or values: packed codes [pages, kv_heads, page, dim / 2] in the layout's memory order, blocks and scales."""
    dev, dim, heads, page = gen.device, case["dim"], case["kv_heads"], case["page"]
    order = (pages, heads, page, dim // 2) if layout == "heads" else (pages, page, heads, dim // 2)
    codes = torch.zeros(order, dtype=torch.uint8, device=dev)
    blocks = torch.zeros((pages, heads, page, dim // 16), dtype=torch.uint8, device=dev)
    scales = torch.ones((pages, heads, page), device=dev)
    codes = codes if layout == "heads" else codes.transpose(1, 2)
    for at in range(0, pages if filled else 0, 1024):
        x = torch.randn((min(1024, pages - at), heads, page, dim), generator=gen, device=dev)
        c, b, s = _quantized(x)
        codes[at:at + 1024], blocks[at:at + 1024], scales[at:at + 1024] = _packed(c), b.view(torch.uint8), s
    return codes, blocks, scales


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(int(seed) * 7919 + 17)
    s = dict(case=case)
    op = case["op"]
    if op in ("linear", "requantize"):
        w = torch.empty((case["n"], case["k"]), device=dev).normal_(generator=gen) * 0.02
        # some channels and inputs weigh more than others, as in trained weights
        w *= torch.exp(0.5 * torch.randn((case["n"], 1), generator=gen, device=dev))
        w *= torch.exp(0.3 * torch.randn((1, case["k"]), generator=gen, device=dev))
    if op == "linear":
        c, b, s["scales"] = _quantized(w)
        s["codes"], s["blocks"] = _packed(c), b.view(torch.uint8)
        del c, b, w
        s["x"] = torch.empty((case["m"], case["k"]), device=dev, dtype=DTYPES[case["dtype"]]).normal_(generator=gen)
        s["bias"] = torch.randn(case["n"], generator=gen, device=dev) if case["bias"] else None
    elif op == "requantize":
        s["w"] = w.to(DTYPES[case["dtype"]])
    elif op == "append":
        tokens, rot, axes, heads, kv = case["tokens"], case["rot"], case["axes"], case["q_heads"], case["kv_heads"]
        s["table"], s["sections"] = _table(rot, dev), _sections(rot, axes)
        s["axis"] = torch.repeat_interleave(torch.arange(axes, device=dev), torch.tensor(s["sections"], device=dev))
        s["positions"] = torch.randint(0, MAX_POS, (axes, tokens), generator=gen, device=dev, dtype=torch.int32)
        row = torch.empty((tokens, heads + 2 * kv, case["dim"]), device=dev, dtype=DTYPES[case["dtype"]])
        row.normal_(generator=gen)
        s["q"], s["k"], s["v"] = row[:, :heads], row[:, heads:heads + kv], row[:, heads + kv:]
        pages = tokens // case["page"] + 3
        s["slots"] = torch.randperm(pages * case["page"], generator=gen, device=dev)[:tokens]
        if tokens > 256:  # a prompt fills whole pages in order, the pages being anywhere
            where = torch.randperm(pages, generator=gen, device=dev)
            at = torch.arange(tokens, device=dev)
            s["slots"] = where[at // case["page"]] * case["page"] + at % case["page"]
        (s["kc"], s["kb"], s["ks"]), (s["vc"], s["vb"], s["vs"]) = (_cache_half(case, pages, gen, False, "heads") for _ in range(2))
    else:
        new, lens = _lengths(case)
        page, heads = case["page"], case["kv_heads"] * case["group"]
        need = [-(-t // page) for t in lens]
        pages = sum(need) + 5
        where = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        col = torch.arange(max(need) + 1, device=dev)
        first = torch.tensor([0] + need, device=dev).cumsum(0)[:-1]
        used = col[None, :] < torch.tensor(need, device=dev)[:, None]
        s["block_table"] = torch.where(used, where[(first[:, None] + col[None, :]).clamp(max=pages - 1)], 0).to(torch.int32).contiguous()
        s["lens"] = torch.tensor(lens, device=dev, dtype=torch.int32)
        s["starts"] = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
        s["new"], s["max_new"], s["max_len"] = new, max(new), max(lens)
        # queries as the leading columns of a fused projection's rows
        row = torch.empty((sum(new), heads + 2 * case["kv_heads"], case["dim"]), device=dev, dtype=DTYPES[case["dtype"]])
        s["q"] = row.normal_(generator=gen)[:, :heads]
        (s["kc"], s["kb"], s["ks"]), (s["vc"], s["vb"], s["vs"]) = (_cache_half(case, pages, gen, True, case["layout"]) for _ in range(2))
        # where each token's row stands in a rectangle of sequences, for the plain form
        s["seq_of"] = torch.repeat_interleave(torch.arange(len(new), device=dev), torch.tensor(new, device=dev))
        s["index_of"] = torch.arange(sum(new), device=dev) - s["starts"].long()[s["seq_of"]]
    if own:
        import fp8_weight_only_gb300 as fw
        s["fw"] = fw
        if op == "append":
            s["rope"] = fw.Rope(s["table"], sections=s["sections"], interleaved=case["pairs"] == "interleaved")
        if op in ("append", "attend"):
            s["cache"] = fw.KVCache(s["kc"], s["vc"], s["ks"], s["vs"], s["kb"], s["vb"])
    return s


# --------------------------------------------------------------- plain forms --

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


def _put(s, name, x):
    """Rows x [tokens, kv_heads, dim] in 32 bits into their slots."""
    page = s["case"]["page"]
    at, off = s["slots"] // page, s["slots"] % page
    c, b, scale = _quantized(x)
    s[name + "c"][at, :, off], s[name + "b"][at, :, off], s[name + "s"][at, :, off] = _packed(c), b.view(torch.uint8), scale


def _gathered(s, name):
    """The cached rows of each sequence in order, [seqs, kv_heads, width * page, dim] in 32 bits."""
    at = s["block_table"].long()
    return _values(s[name + "c"][at], s[name + "b"][at], s[name + "s"][at]).transpose(1, 2).flatten(2, 3)


def _attend(s):
    case = s["case"]
    heads, group, dim = case["kv_heads"], case["group"], case["dim"]
    seqs, most = case["seqs"], s["max_new"]
    k = _gathered(s, "k")
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
    out = weight.view(seqs, heads, most * group, -1) @ _gathered(s, "v")
    out = out.view(seqs, heads, most, group, dim) / torch.where(total == 0, torch.ones_like(total), total)
    out = out.permute(0, 2, 1, 3, 4).reshape(seqs, most, heads * group, dim)
    return out[s["seq_of"], s["index_of"]].to(s["q"].dtype)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        fw = s["fw"]
        if op == "linear":
            return fw.linear_fp4(s["x"], s["codes"], s["blocks"], s["scales"], s["bias"])
        if op == "requantize":
            codes, blocks, scales = fw.quantize_fp4(s["w"])
            return dict(w=fw.dequantize_fp4(codes, blocks, scales, DTYPES[case["out"]]), blocks=blocks.view(torch.float8_e4m3fn),
                        scales=scales)
        if op == "append":
            q = fw.rope_append(s["q"], s["k"], s["v"], s["slots"], s["cache"], s["positions"], s["rope"])
            # the cache as the values that it stands for
            return dict(q=q, k=fw.dequantize_fp4(s["kc"], s["kb"], s["ks"], torch.bfloat16),
                        v=fw.dequantize_fp4(s["vc"], s["vb"], s["vs"], torch.bfloat16))
        return fw.paged_attention(s["q"], s["cache"], s["block_table"], s["lens"],
                                  starts=s["starts"] if case["new_hi"] > 1 else None, window=case["window"],
                                  max_new=s["max_new"], max_len=s["max_len"])
    if op == "linear":
        y = s["x"].float() @ _values(s["codes"], s["blocks"], s["scales"]).t()
        return (y if s["bias"] is None else y + s["bias"]).to(s["x"].dtype)
    if op == "requantize":
        codes, blocks, scales = _quantized(s["w"].float())
        return dict(w=_values(_packed(codes), blocks.view(torch.uint8), scales).to(DTYPES[case["out"]]), blocks=blocks, scales=scales)
    if op == "append":
        _put(s, "k", _turn(s["k"], s))
        _put(s, "v", s["v"].float())
        return dict(q=_turn(s["q"], s).to(s["q"].dtype), k=_values(s["kc"], s["kb"], s["ks"]).bfloat16(),
                    v=_values(s["vc"], s["vb"], s["vs"]).bfloat16())
    return _attend(s)


# ---------------------------------------------------------------------- work --

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
    op = case["op"]
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * (k // 2 + k // 16 + 4 + (4 if case["bias"] else 0)) + 2 * m * (n + k), "flops": 2 * m * n * k}
    if op == "requantize":
        n, k = case["n"], case["k"]
        held = n * (k // 2 + k // 16 + 4)
        each = {"f32": 4, "bf16": 2, "f16": 2}
        # the weight read, codes written and read again, the values written
        return {"bytes": n * k * (each[case["dtype"]] + each[case["out"]]) + 2 * held, "flops": 5 * n * k}
    if op == "append":
        tokens, heads, kv, dim = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        row = dim // 2 + dim // 16 + 4
        slots = (tokens // case["page"] + 3) * case["page"] * kv
        rows = min(MAX_POS, tokens * case["axes"])
        # queries and the new rows read and written, and the cache read back as 16-bit values
        return {"bytes": 4 * tokens * heads * dim + 2 * tokens * kv * (2 * dim + row) + (4 * case["axes"] + 8) * tokens +
                4 * rows * case["rot"] // case["axes"] + 2 * slots * (row + 2 * dim),
                "flops": 3 * tokens * (heads + kv) * case["rot"] + 10 * tokens * kv * dim}
    seen, read = _pairs(case)
    heads, dim = case["kv_heads"] * case["group"], case["dim"]
    each = 2 * (dim // 2 + dim // 16 + 4)
    return {"bytes": read * case["kv_heads"] * each + 4 * sum(_lengths(case)[0]) * heads * dim, "flops": 4 * seen * heads * dim}


# --------------------------------------------------------------------- exact --

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _read(codes, blocks, scales):
    """The values of packed rows in 64 bits."""
    k = 2 * codes.shape[-1]
    at = torch.arange(k, device=codes.device)
    nibble = codes.long()[..., at // 2] >> (4 * (at % 2)) & 15
    mag = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)[nibble & 7]
    return torch.where(nibble > 7, -mag, mag) * blocks.view(torch.float8_e4m3fn).double()[..., at // 16] * scales.double()[..., None]


def _statistics(x):
    """The blocks and scales of rows in 64 bits."""
    top = x.abs().max(-1).values
    scales = torch.where(top > 0, (top / 2688).clamp(min=2.0 ** -126), torch.ones_like(top))
    parts = (x / scales[..., None]).reshape(*x.shape[:-1], -1, 16)
    return (parts.abs().max(-1).values / 6).float().clamp(max=448).to(torch.float8_e4m3fn).double(), scales


def exact(case, seed):
    """The case's outputs in 64 bits from the definition: complex turns, and one softmax for each sequence and head."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        x, y = s["x"].double(), []
        for at in range(0, case["n"], 2048):
            rows = slice(at, at + 2048)
            y.append(x @ _read(s["codes"][rows], s["blocks"][rows], s["scales"][rows]).t())
        y = torch.cat(y, 1)
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "requantize":
        parts = [_statistics(s["w"][at:at + 1024].double()) for at in range(0, case["n"], 1024)]
        b, sc = (torch.cat(p) for p in zip(*parts))
        # 16-bit weights lie on the middle of two codes often, where the side taken is a matter of the
        # steps that the form prescribes: the codes have no value of their own in 64 bits
        return dict(w=None, blocks=b, scales=sc)
    if op == "append":
        rot = case["rot"]
        half = rot // 2

        def turned(x):
            x = x.double().clone()
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

        return dict(q=turned(s["q"]), k=None, v=None)  # as above
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
            k, v = (_read(s[c + "c"][pages, h], s[c + "b"][pages, h], s[c + "s"][pages, h]).flatten(0, 1)[:t] for c in "kv")
            for g in range(h * case["group"], (h + 1) * case["group"]):
                q = s["q"][starts[b]:starts[b + 1], g].double()
                z = (q @ k.t()) / math.sqrt(case["dim"])
                out[starts[b]:starts[b + 1], g] = torch.softmax(z.masked_fill_(hidden, float("-inf")), -1) @ v
    return out
