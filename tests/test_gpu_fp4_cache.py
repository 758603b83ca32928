"""GPU tests of the 4-bit cache: rows appended bit for bit as the rule gives
them, and attention against 64 bits on the values that the cache stands for
(bounds: attention_reference.py; the products of a code and its block's scale are
exact, so the form adds nothing to them).

The weights are fp16 here whatever the activations' type, so the bounds of bf16 get
what fp16 takes below its normal numbers, too:  keys 2^-32 max|v|.
  A weight times its slot's scale, p_j s_j, is taken 2^7 times as large as its
  reference, which lies at most 2^8 under the largest and never above it (but by
  fp32 roundings): the largest is 2^7 in fp16 at least.  Below 2^-14 fp16 rounds by
  2^-25 at most, 2^-32 of that largest.  Row j's values are s_j times 2688 at most,
  and its largest is that (the rule's scale), so a weight's error adds at most
  2^-32 max_j(p_j s_j) 2688 <= 2^-32 max|v| to an output (sum of the p at least the
  largest), and `keys` weights that many times as much."""
import numpy as np
import pytest

from tests import fp4_reference as R
from tests.attention_reference import attend, bits, check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_weight_only_gb300 as fw  # noqa: E402
from tests.test_gpu_rope import rows, table, turn  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
POISON = 0x7FC1


# ------------------------------------------------------------------ append --

def bound(tol, v, length, dtype):
    return tol + (length * 2.0 ** -32 * float(v.abs().max()) if dtype == "bf16" and length else 0.0)


def empty_cache(pages, kv, page, dim, layout, fill=0xA5):
    shape = (pages, kv, page, dim // 2) if layout == "heads" else (pages, page, kv, dim // 2)
    view = (lambda t: t) if layout == "heads" else (lambda t: t.transpose(1, 2))
    k, v = (view(torch.full(shape, fill, dtype=torch.uint8, device=DEV)) for _ in range(2))
    kb, vb = (torch.full((pages, kv, page, dim // 16), fill, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((pages, kv, page), -3.0, device=DEV) for _ in range(2))
    return fw.KVCache(k, v, ks, vs, kb, vb)


def held(cache):
    return [t.cpu().numpy().copy() for t in (cache.k, cache.k_blocks, cache.k_scales, cache.v, cache.v_blocks, cache.v_scales)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
@pytest.mark.parametrize("tokens,heads,kv,dim,rot,sections,interleaved", [
    (1, 4, 1, 32, 32, [16], False), (1, 32, 8, 128, 128, [64], False), (5, 3, 3, 64, 16, [8], False), (9, 2, 2, 64, 48, [24], False),
    (33, 8, 2, 96, 80, [13, 27], False), (40, 4, 4, 96, 96, [16, 16, 16], True), (200, 4, 2, 128, 64, [32], True),
    (700, 8, 4, 128, 112, [20, 20, 16], False), (3000, 2, 1, 32, 16, [8], False)])
def test_append(tokens, heads, kv, dim, rot, sections, interleaved, layout, dtype):
    page = 16
    pages = tokens // page + 3
    row = rows(tokens + dim, tokens, heads + 2 * kv, dim, dtype)
    q, k, v = row[:, :heads], row[:, heads:heads + kv], row[:, heads + kv:]
    if tokens > 4:
        k[2], v[3] = 0.0, 0.0
    tab = table(3000, rot)
    pos = torch.randint(0, 3000, (len(sections), tokens), device=DEV, dtype=torch.int32)
    slots = torch.randperm(pages * page, device=DEV)[:tokens]
    if tokens > 8:
        slots[7] = -1                               # a padded token
    cache = empty_cache(pages, kv, page, dim, layout)
    want = held(cache)
    out = fw.rope_append(q, k, v, slots, cache, pos, fw.Rope(tab, interleaved=interleaved, sections=sections))
    assert fw.device_error() == 0
    tq = turn(q.cpu().float(), pos, tab, sections, interleaved)
    assert np.array_equal(bits(out.cpu()), bits(tq.to(DT[dtype])))
    both = (turn(k.cpu().float(), pos, tab, sections, interleaved).numpy(), v.cpu().float().numpy())
    s = slots.cpu().numpy()
    keep = s >= 0
    at, off = s[keep] // page, s[keep] % page
    for i, x in enumerate(both):
        got = R.quantize(x[keep])
        for j in range(3):
            want[3 * i + j][at, :, off] = got[j]
    for a, b in zip(held(cache), want):             # every other slot as it was
        assert np.array_equal(a.view(np.uint8), b.view(np.uint8))


def test_append_without_rotation_or_queries():
    k, v = rows(1, 6, 2, 64, "bf16"), rows(2, 6, 2, 64, "bf16")
    cache = empty_cache(2, 2, 16, 64, "heads")
    assert fw.rope_append(None, k, v, torch.arange(6, device=DEV), cache) is None
    got = R.quantize(k.cpu().float().numpy())
    assert np.array_equal(cache.k[0, :, :6].cpu().numpy(), got[0].swapaxes(0, 1))
    assert np.array_equal(cache.k_blocks[0, :, :6].cpu().numpy(), got[1].swapaxes(0, 1))
    assert np.array_equal(cache.k_scales[0, :, :6].cpu().numpy(), got[2].swapaxes(0, 1))


def test_a_slot_beyond_the_cache_is_recorded():
    k, v = rows(1, 2, 2, 64, "bf16"), rows(2, 2, 2, 64, "bf16")
    cache = empty_cache(2, 2, 16, 64, "heads")
    before = held(cache)
    fw.rope_append(None, k, v, torch.tensor([32, 10 ** 12], device=DEV), cache)
    assert fw.device_error() != 0 and fw.device_error() == 0
    assert all(np.array_equal(a.view(np.uint8), b.view(np.uint8)) for a, b in zip(held(cache), before))


# --------------------------------------------------------------- attention --

def run(new, lens, kv_heads, group, dim, page, dtype="bf16", layout="heads", window=0, seed=1, growth=0.0, starts=None, max_new=0,
        max_len=0, q_scale=1.0, change=None):
    paged = R.Paged4(torch, fw, seed, lens, kv_heads, dim, page, layout, growth=growth, change=change)
    tokens, heads = sum(new), kv_heads * group
    g = torch.Generator(DEV)
    g.manual_seed(seed + 100)
    # queries inside wider rows, outputs inside a poisoned buffer with wider rows
    q = (torch.randn((tokens, heads + 2, dim), generator=g, device=DEV) * q_scale).to(DT[dtype])[:, :heads]
    buf = torch.empty((tokens + 2, heads + 1, dim), dtype=DT[dtype], device=DEV)
    buf.view(torch.int16).fill_(POISON)
    out = buf[1:-1, :heads]
    first = np.concatenate([[0], np.cumsum(new)])
    if starts is None and any(n != 1 for n in new):
        starts = torch.tensor(first, dtype=torch.int32, device=DEV)
    fw.paged_attention(q, paged.cache, paged.table, paged.lens_t, starts=starts, window=window, max_new=max_new, max_len=max_len, out=out)
    assert fw.device_error() == 0
    rest = buf.clone()
    rest[1:-1, :heads].view(torch.int16).fill_(POISON)
    assert bool((rest.view(torch.int16) == POISON).all()), "written outside the output"
    for b, n in enumerate(new):
        k, v = paged.rows[b]
        want, tol = attend(torch, q[first[b]:first[b + 1]].double(), k, v, n, lens[b], dim ** -0.5, window, dtype)
        check(torch, out[first[b]:first[b + 1]], want, bound(tol, v, lens[b], dtype))
    return q, paged, out


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 33, 127, 128, 129, 640])
def test_one_sequence(length, dim, dtype):
    run([1], [length], 2, 4, dim, 16, dtype)


@pytest.mark.parametrize("group", [1, 3, 7, 8, 9, 16, 17, 48, 49, 130, 300])
@pytest.mark.parametrize("dim", [64, 128])
def test_query_heads_to_a_key_head(group, dim):
    run([1, 1], [200, 77], 1, group, dim, 16)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
@pytest.mark.parametrize("dim", [32, 96, 128])
def test_page_sizes_and_memory_orders(page, layout, dim):
    run([1, 1, 1], [1, 700, page + 1], 3, 2, dim, page, "f16", layout)
    run([70, 60], [700, page + 60], 3, 2, dim, page, "bf16", layout)


@pytest.mark.parametrize("group", [4, 20])
def test_ragged_batch_with_empty_sequences(group):
    lens = [0, 1, 15, 16, 17, 1000, 0, 129, 2049, 64, 0]
    _, _, out = run([1] * len(lens), lens, 4, group, 128, 16)
    for b in (0, 6, 10):
        assert not out[b].any()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("length,kv_heads,group", [(4000, 1, 8), (9001, 2, 8), (40007, 1, 4), (2300, 8, 8), (9001, 1, 64)])
def test_long_cache_split_over_a_cluster(length, kv_heads, group, dtype):
    run([1], [length], kv_heads, group, 128, 64, dtype, seed=3)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("new,length", [(2, 2), (12, 31), (13, 300), (33, 33), (64, 64), (65, 1000), (257, 300), (700, 700)])
def test_chunks(new, length, dim, dtype):
    run([new], [length], 1, 4, dim, 16, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_mixed_batch_and_window(dtype):
    new, lens = [1, 200, 1, 1, 65, 3], [0, 450, 1, 3001, 65, 90]
    run(new, lens, 2, 4, 128, 16, dtype, max_new=200, max_len=3001)
    run(new, lens, 2, 4, 64, 32, dtype, window=100, max_new=200)
    run([1] * 4, [0, 300, 5000, 20], 2, 4, 128, 32, dtype, window=77)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new", [1, 40])
def test_scores_that_grow(new, dtype):
    run([new], [3000], 1, 8, 128, 16, dtype, growth=6.0, q_scale=2.0)


def zero_rows(at):
    def change(b, x):
        x[0, at] *= 8.0                             # the largest scores at rows of zeros
        x[1, at] = 0.0
        x[1, :at] *= 1e-3
        x[1, at + 1:] *= 1e-3
    return change


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new", [1, 60])
def test_rows_of_zeros_do_not_hide_small_values(new, dtype):
    run([new], [400], 1, 4, 64, 16, dtype, change=zero_rows(130))


@pytest.mark.parametrize("new,window", [(4, 0), (60, 0), (200, 33)])
def test_bf16_queries_of_every_magnitude(new, window):
    """Heads and tokens from 2^-120 to 2^6 times as large as others, and values far below their row's largest."""
    paged = R.Paged4(torch, fw, 5, [700], 2, 128, 16, "heads")
    g = torch.Generator(DEV)
    g.manual_seed(9)
    q = torch.randn((new, 8, 128), generator=g, device=DEV)
    q *= torch.exp2(torch.randint(-12, 1, q.shape, generator=g, device=DEV).float())
    q *= torch.exp2(torch.linspace(-120, 6, new * 8, device=DEV)).view(new, 8, 1)[torch.randperm(new, generator=g, device=DEV)]
    q[0, 1] = 0.0
    q = q.bfloat16()
    starts = torch.tensor([0, new], dtype=torch.int32, device=DEV)
    got = fw.paged_attention(q, paged.cache, paged.table, paged.lens_t, starts=starts, window=window)
    assert fw.device_error() == 0
    want, tol = attend(torch, q.double(), *paged.rows[0], new, 700, 128 ** -0.5, window, "bf16")
    check(torch, got, want, bound(tol, paged.rows[0][1], 700, "bf16"))


@pytest.mark.parametrize("new", [1, 30])
def test_a_query_that_is_not_finite_reaches_its_row_alone(new):
    q, paged, out = run([new, new], [90, 300], 2, 4, 128, 16)
    bad = q.clone()
    bad[new, 3, 7] = float("nan")
    starts = torch.tensor([0, new, 2 * new], dtype=torch.int32, device=DEV)
    got = fw.paged_attention(bad, paged.cache, paged.table, paged.lens_t, starts=starts)
    assert bool(torch.isnan(got[new, 3]).all())
    got[new, 3] = out[new, 3]
    assert torch.equal(got, out)


def test_pages_past_four_gib():
    # offsets beyond 32 bits: 2^27 bytes a page stride
    pages, kv, page, dim = 40, 1, 16, 64
    stride = 1 << 27
    store = torch.empty(pages * stride, dtype=torch.uint8, device=DEV)
    k = torch.as_strided(store, (pages, kv, page, dim // 2), (stride, page * dim // 2, dim // 2, 1))
    v = torch.as_strided(store, (pages, kv, page, dim // 2), (stride, page * dim // 2, dim // 2, 1), 4096)
    rng = np.random.default_rng(1)
    both = [R.quantize(rng.standard_normal((pages, kv, page, dim)).astype(np.float32)) for _ in range(2)]
    k.copy_(torch.from_numpy(both[0][0]))
    v.copy_(torch.from_numpy(both[1][0]))
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    cache = fw.KVCache(k, v, d(both[0][2]), d(both[1][2]), d(both[0][1]), d(both[1][1]))
    order = torch.randperm(pages, device=DEV).int()[None]
    length = pages * page - 3
    for new in (1, 50):
        q = torch.randn((new, 2, dim), device=DEV).bfloat16()
        got = fw.paged_attention(q, cache, order, torch.tensor([length], dtype=torch.int32, device=DEV),
                                 starts=torch.tensor([0, new], dtype=torch.int32, device=DEV))
        assert fw.device_error() == 0
        kk, vv = (d(R.values(*b))[order[0].long()].transpose(1, 2).flatten(0, 1)[:length] for b in both)
        want, tol = attend(torch, q.double(), kk, vv, new, length, dim ** -0.5, 0, "bf16")
        check(torch, got, want, bound(tol, vv, length, "bf16"))


def test_a_page_outside_the_cache_is_recorded():
    _, paged, _ = run([1], [100], 1, 2, 64, 16)
    paged.table[0, 3] = 10 ** 6
    for group, new in ((2, 1), (2, 100)):
        q = torch.randn((new, group, 64), device=DEV).bfloat16()
        got = fw.paged_attention(q, paged.cache, paged.table, paged.lens_t, starts=torch.tensor([0, new], dtype=torch.int32, device=DEV))
        assert fw.device_error() != 0 and fw.device_error() == 0
        assert bool(torch.isfinite(got).all())


# ---------------------------------------------------------------- together --

def decoded(graph, steps=60, group=4, seqs=5):
    """A decoder block's attention half on 4-bit weights and a 4-bit cache, step by step."""
    kv, dim, page, width, hidden = 2, 128, 16, 6, 512
    g = torch.Generator(DEV)
    g.manual_seed(4)
    heads = kv * group
    wq = fw.quantize_fp4(torch.randn(((heads + 2 * kv) * dim, hidden), generator=g, device=DEV) * 0.05)
    wo = fw.quantize_fp4(torch.randn((hidden, heads * dim), generator=g, device=DEV) * 0.05)
    cache = empty_cache(seqs * width, kv, page, dim, "heads", fill=0)
    pages = torch.randperm(seqs * width, generator=g, device=DEV).int().view(seqs, width)
    rope = fw.Rope(table(steps, dim))
    at = torch.arange(steps, device=DEV)
    slots = (pages.long()[:, at // page] * page + at % page).t().contiguous()
    lens = (at[:, None] + 1).int().expand(steps, seqs).contiguous()
    positions = at[:, None].int().expand(steps, seqs).contiguous()
    x = torch.randn((seqs, hidden), generator=g, device=DEV).bfloat16()

    def go(wait):
        y, outs = x, []
        sync = torch.cuda.synchronize if wait else (lambda: None)
        for i in range(steps):
            fused = fw.linear_fp4(y, *wq).view(seqs, heads + 2 * kv, dim)
            sync()
            q, k, v = fused.split([heads, kv, kv], 1)
            q = fw.rope_append(q, k, v, slots[i], cache, positions[i], rope)
            sync()
            o = fw.paged_attention(q, cache, pages, lens[i])
            sync()
            y = fw.linear_fp4(o.view(seqs, heads * dim), *wo)
            sync()
            outs.append(y)
        return torch.stack(outs)

    torch.cuda.synchronize()
    if not graph:
        return go(True)
    held_graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(held_graph):
        out = go(False)
    held_graph.replay()
    torch.cuda.synchronize()
    return out.clone()


def test_a_block_in_four_bits_gives_in_a_graph_what_its_calls_give():
    a, b = decoded(False), decoded(True)
    assert bool(torch.isfinite(a).all()) and a.float().abs().max() > 0
    assert torch.equal(a, b)
    assert fw.device_error() == 0
