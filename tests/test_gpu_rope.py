"""GPU tests of fp8w_rope and fp8w_rope_append: bit for bit against the same
products and sums in fp32 (each rounded once, then once to the output type),
within one rounding of the rotation in 64 bits, and e4m3 codes and scales
equal to the oracle quantiser's on the fp32 rows."""
import numpy as np
import pytest

import oracle
from tests.attention_reference import ROUND, bits

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_weight_only_gb300 as fw  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def table(max_pos, rot):
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, device=DEV, dtype=torch.float64)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def turn(x, positions, tab, sections, interleaved):
    """The rotation in x's own type (fp32: each product and sum rounded; fp64), on the CPU."""
    x, pos, tab = x.clone(), positions.cpu().long(), tab.cpu().to(x.dtype)
    half = tab.shape[1] // 2
    axis = np.repeat(np.arange(len(sections)), sections)
    for i in range(half):
        row = tab[pos[axis[i]]]
        c, s = row[:, i][:, None], row[:, half + i][:, None]
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = x[..., ia].clone(), x[..., ib].clone()
        x[..., ia] = a * c - b * s
        x[..., ib] = b * c + a * s
    return x


def rows(seed, tokens, heads, dim, dtype, extra=0):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    return torch.randn((tokens, heads + extra, dim), generator=g, device=DEV).to(DT[dtype])[:, :heads]


def near(got, want, dtype):
    """One rounding to the type after fp32 steps (three roundings of 2^-24 of |a c| + |b s| <= 16 here)."""
    tol = ROUND[dtype] * want.abs() + 3 * 2.0 ** -24 * 16 + (2.0 ** -25 if dtype == "f16" else 0.0)
    assert bool(((got.cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,rot,sections", [
    (1, 1, 16, 16, [8]), (3, 5, 64, 32, [16]), (7, 40, 128, 128, [64]), (33, 3, 80, 80, [13, 27]),
    (50, 2, 128, 96, [16, 20, 12]), (5, 9, 256, 256, [50, 0, 70, 8]), (400, 6, 96, 96, [16, 16, 16])])
def test_rope(tokens, heads, dim, rot, sections, interleaved, dtype):
    x = rows(7, tokens, heads, dim, dtype, extra=3)
    tab = table(5000, rot)
    pos = torch.randint(0, 5000, (len(sections), tokens), device=DEV, dtype=torch.int32)
    spec = fw.Rope(tab, interleaved=interleaved, sections=sections)
    buf = torch.full((tokens + 2, heads + 1, dim), -7.0, dtype=DT[dtype], device=DEV)
    got = fw.rope(x, pos, spec, out=buf[1:-1, :heads])
    assert fw.device_error() == 0
    want = turn(x.cpu().float(), pos, tab, sections, interleaved).to(DT[dtype])
    assert np.array_equal(bits(got.cpu()), bits(want))
    near(got, turn(x.cpu().double(), pos, tab, sections, interleaved), dtype)
    rest = buf.clone()
    rest[1:-1, :heads] = -7.0
    assert bool((rest == -7.0).all())
    # in place, the rows' own strides
    y = x
    fw.rope(y, pos, spec, out=y)
    assert np.array_equal(bits(y.cpu()), bits(want))


def test_position_zero_is_the_identity_and_a_turn_keeps_length():
    x = rows(3, 20, 4, 64, "f16")
    tab = table(100, 64)
    zero = torch.zeros(20, dtype=torch.int32, device=DEV)
    assert np.array_equal(bits(fw.rope(x, zero, fw.Rope(tab))), bits(x))
    pos = torch.arange(20, dtype=torch.int32, device=DEV)
    y = fw.rope(x, pos, fw.Rope(tab)).double()
    a, b = x.double().pow(2).sum(-1), y.pow(2).sum(-1)
    assert float(((a - b).abs() / a).max()) <= 2 * 2 ** -11 + 1e-6


def test_positions_outside_the_table_are_moved_to_its_ends_and_recorded():
    x = rows(3, 4, 2, 64, "bf16")
    tab = table(50, 64)
    got = fw.rope(x, torch.tensor([-3, 50, 49, 2 ** 31 - 1], dtype=torch.int32, device=DEV), fw.Rope(tab))
    assert fw.device_error() == 6006 and fw.device_error() == 0
    want = fw.rope(x, torch.tensor([0, 49, 49, 49], dtype=torch.int32, device=DEV), fw.Rope(tab))
    assert np.array_equal(bits(got), bits(want)) and fw.device_error() == 0


def make_cache(pages, kv, page, dim, dtype, codes, layout):
    shape = (pages, kv, page, dim) if layout == "heads" else (pages, page, kv, dim)
    k = torch.full(shape, 0x55 if codes else 3.0, dtype=torch.uint8 if codes else DT[dtype], device=DEV)
    k = k if layout == "heads" else k.transpose(1, 2)
    ks = torch.full((pages, kv, page), -1.0, device=DEV) if codes else None
    v = torch.empty_strided(k.shape, k.stride(), dtype=k.dtype, device=DEV).copy_(k)
    return fw.KVCache(k, v, ks, None if ks is None else ks.clone())


@pytest.mark.parametrize("dtype,codes", [("bf16", False), ("f16", False), ("bf16", True), ("f16", True)])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
@pytest.mark.parametrize("tokens,q_heads,kv,dim,rot,sections,interleaved,page", [
    (1, 32, 8, 128, 128, [64], False, 16), (5, 3, 1, 16, 16, [8], True, 16), (130, 6, 3, 80, 48, [10, 14], False, 32),
    (700, 8, 2, 96, 96, [16, 16, 16], True, 256), (67, 5, 5, 64, 0, None, False, 64)])
def test_rope_append(tokens, q_heads, kv, dim, rot, sections, interleaved, page, layout, dtype, codes):
    fused = rows(11, tokens, q_heads + 2 * kv, dim, dtype)
    q, k, v = fused[:, :q_heads], fused[:, q_heads:q_heads + kv], fused[:, q_heads + kv:]
    if tokens > 3:
        k[2], v[3] = 0, 0   # all-zero rows take scale 1
    pages = tokens // page + 3
    cache = make_cache(pages, kv, page, dim, dtype, codes, layout)
    slots = torch.randperm(pages * page, device=DEV)[:tokens]
    if tokens > 4:
        slots[4] = -1       # a padded token
    spec = pos = None
    kr, qr, vr = k.cpu().float(), q.cpu().float(), v.cpu().float()
    if rot:
        tab = table(3001, rot)
        pos = torch.randint(0, 3001, (len(sections), tokens), device=DEV, dtype=torch.int32)
        spec = fw.Rope(tab, interleaved=interleaved, sections=sections)
        kr, qr = turn(kr, pos, tab, sections, interleaved), turn(qr, pos, tab, sections, interleaved)
    before = [t.clone() for t in (cache.k, cache.v)]
    got = fw.rope_append(q, k, v, slots, cache, pos, spec)
    assert fw.device_error() == 0
    assert np.array_equal(bits(got.cpu()), bits(qr.to(DT[dtype])))
    for name, x, was in (("k", kr, before[0]), ("v", vr, before[1])):
        held, want = getattr(cache, name).cpu(), was.cpu()
        sc = want_s = None
        if codes:
            sc, want_s = getattr(cache, name + "_scales").cpu(), torch.full((pages, kv, page), -1.0)
            code, scale = oracle.quantize(x.reshape(tokens * kv, dim).numpy())
            code, scale = torch.from_numpy(code).view(tokens, kv, dim), torch.from_numpy(scale).view(tokens, kv)
        for t, s in enumerate(slots.tolist()):
            if s < 0:
                continue
            if codes:
                want[s // page, :, s % page], want_s[s // page, :, s % page] = code[t], scale[t]
            else:
                want[s // page, :, s % page] = x[t].to(DT[dtype])
        if codes:
            assert torch.equal(held, want) and np.array_equal(bits(sc), bits(want_s))
        else:
            assert np.array_equal(bits(held), bits(want))


def test_append_without_queries_and_beyond_the_cache():
    cache = make_cache(2, 1, 16, 64, "bf16", False, "heads")
    k, v = rows(1, 4, 1, 64, "bf16"), rows(2, 4, 1, 64, "bf16")
    before = cache.k.clone()
    assert fw.rope_append(None, k, v, torch.tensor([32, 2 ** 60, -5, 31], device=DEV), cache) is None
    assert fw.device_error() == 6006 and fw.device_error() == 0
    before[1, 0, 15] = k[3, 0]
    assert torch.equal(cache.k, before)


def test_append_to_pages_beyond_4_gib():
    stride = 1 << 31
    big = torch.zeros(3 * stride, dtype=torch.uint8, device=DEV)
    k, v = (torch.as_strided(big, (3, 1, 16, 64), (stride, 1024, 64, 1), off) for off in (0, 1 << 20))
    ks, vs = torch.zeros((3, 1, 16), device=DEV), torch.zeros((3, 1, 16), device=DEV)
    x = rows(1, 2, 1, 64, "f16")
    fw.rope_append(None, x, x, torch.tensor([2 * 16 + 5, 0], device=DEV), fw.KVCache(k, v, ks, vs))
    code, scale = oracle.quantize(x.float().cpu().view(2, 64).numpy())
    assert np.array_equal(v[2, 0, 5].cpu().numpy(), code[0]) and float(vs[2, 0, 5]) == scale[0]
    assert np.array_equal(k[0, 0, 0].cpu().numpy(), code[1])


def test_in_place_queries_on_another_stream_and_in_a_graph():
    cache = make_cache(4, 2, 16, 128, "bf16", True, "tokens")
    fused = rows(5, 40, 8, 128, "bf16")
    q, k, v = fused[:, :4], fused[:, 4:6], fused[:, 6:]
    pos, spec, slots = torch.arange(40, dtype=torch.int32, device=DEV), fw.Rope(table(64, 128)), torch.arange(40, device=DEV)
    want = bits(fw.rope_append(q, k, v, slots, cache, pos, spec))
    codes = cache.k.clone()
    cache.k.fill_(0x55)   # as before the call
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fw.rope_append(q, k, v, slots, cache, pos, spec, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(bits(out), want) and torch.equal(cache.k, codes)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fw.rope_append(q, k, v, slots, cache, pos, spec, out=q)
    side.synchronize()
    assert np.array_equal(bits(q), want)
