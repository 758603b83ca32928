"""GPU tests of fp8w_paged_attention against attention in 64 bits: lengths of
zero and one, pages that end inside a tile, sequences split over a cluster,
windows, rows that see nothing, NaN in every slot that no sequence owns."""
import numpy as np
import pytest

from tests.attention_reference import Paged, attend, bits, check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_weight_only_gb300 as fw  # noqa: E402

DEV = torch.device("cuda:0")
POISON = 0x7FC1


def run(new, lens, kv_heads, group, dim, page, dtype="bf16", codes=False, layout="heads", window=0, seed=1, growth=0.0,
        starts=None, max_new=0, max_len=0, scale=None, q_scale=1.0):
    paged = Paged(torch, fw, seed, lens, kv_heads, dim, page, dtype, codes, layout, growth=growth)
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float16
    tokens, heads = sum(new), kv_heads * group
    g = torch.Generator(DEV)
    g.manual_seed(seed + 100)
    # queries inside wider rows, outputs inside a poisoned buffer with wider rows
    q = (torch.randn((tokens, heads + 2, dim), generator=g, device=DEV) * q_scale).to(tdt)[:, :heads]
    buf = torch.empty((tokens + 2, heads + 1, dim), dtype=tdt, device=DEV)
    buf.view(torch.int16).fill_(POISON)
    out = buf[1:-1, :heads]
    first = np.concatenate([[0], np.cumsum(new)])
    if starts is None and any(n != 1 for n in new):
        starts = torch.tensor(first, dtype=torch.int32, device=DEV)
    fw.paged_attention(q, paged.cache, paged.table, paged.lens_t, starts=starts, window=window, max_new=max_new,
                       max_len=max_len, scale=scale, out=out)
    assert fw.device_error() == 0
    rest = buf.clone()
    rest[1:-1, :heads].view(torch.int16).fill_(POISON)
    assert bool((rest.view(torch.int16) == POISON).all()), "written outside the output"
    for b, n in enumerate(new):
        k, v = paged.rows[b]
        want, tol = attend(torch, q[first[b]:first[b + 1]].double(), k, v, n, lens[b], dim ** -0.5 if scale is None else scale,
                           window, dtype)
        check(torch, out[first[b]:first[b + 1]], want, tol)
    return q, paged, out


# ---------------------------------------------------------- single tokens --

@pytest.mark.parametrize("dtype,codes", [("bf16", False), ("f16", False), ("bf16", True), ("f16", True)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("length", [1, 2, 127, 128, 129, 640])
def test_one_sequence(length, dim, dtype, codes):
    run([1], [length], 2, 4, dim, 16, dtype, codes)


@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 16, 33, 128, 129, 256, 300])
def test_query_heads_to_a_key_head(group):
    run([1, 1], [200, 77], 1, group, 64, 16)


@pytest.mark.parametrize("dim", [16, 32, 48, 80, 96, 112])
@pytest.mark.parametrize("codes", [False, True])
def test_head_sizes_between_the_tile_widths(dim, codes):
    run([1, 1, 1], [300, 5, 128], 2, 4, dim, 16, "bf16", codes)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_page_sizes_and_memory_orders(page, codes, layout):
    run([1, 1, 1], [1, 700, page + 1], 3, 2, 128, page, "f16", codes, layout)


@pytest.mark.parametrize("codes", [False, True])
def test_ragged_batch_with_empty_sequences(codes):
    lens = [0, 1, 15, 16, 17, 1000, 0, 129, 2049, 64, 0]
    _, _, out = run([1] * len(lens), lens, 4, 4, 128, 16, "bf16", codes)
    for b in (0, 6, 10):
        assert not out[b].any()


@pytest.mark.parametrize("dtype,codes", [("bf16", False), ("f16", True)])
@pytest.mark.parametrize("length,kv_heads", [(4000, 1), (9001, 2), (40007, 1), (2300, 8)])
def test_long_cache_split_over_a_cluster(length, kv_heads, dtype, codes):
    run([1], [length], kv_heads, 8, 128, 64, dtype, codes, seed=3)


@pytest.mark.parametrize("max_len", [0, 1, 5000, 10 ** 9])
def test_the_length_hint_changes_no_result_beyond_rounding(max_len):
    run([1, 1], [5000, 33], 1, 4, 128, 16, max_len=max_len)


# ------------------------------------------------------------------ chunks --

@pytest.mark.parametrize("dtype,codes", [("bf16", False), ("f16", False), ("bf16", True), ("f16", True)])
@pytest.mark.parametrize("new,length", [(2, 2), (31, 31), (32, 300), (33, 33), (64, 64), (65, 1000), (257, 300), (700, 700)])
def test_chunks(new, length, dtype, codes):
    run([new], [length], 1, 4, 128, 16, dtype, codes)


@pytest.mark.parametrize("dtype,codes", [("bf16", False), ("f16", True)])
@pytest.mark.parametrize("dim", [64, 128])
def test_long_chunks(dim, dtype, codes):
    run([513, 300], [7000, 5001], 2, 4, dim, 32, dtype, codes)


@pytest.mark.parametrize("group", [1, 3, 5, 8])
@pytest.mark.parametrize("dim", [64, 80])
def test_chunk_rows_of_odd_groups(group, dim):
    run([301, 1, 77], [301, 900, 500], 2, group, dim, 32, "f16")


@pytest.mark.parametrize("codes", [False, True])
def test_two_row_tiles_split_over_a_cluster(codes):
    run([64], [6000], 1, 4, 128, 16, "bf16", codes)
    run([300], [9000], 1, 1, 64, 16, "bf16", codes)


def test_mixed_batch_with_hints():
    new, lens = [1, 200, 1, 1, 65, 3], [0, 450, 1, 3001, 65, 90]
    run(new, lens, 2, 4, 128, 16, max_new=200, max_len=3001)


def test_sequences_without_new_tokens():
    run([3, 0, 130, 0, 0, 1, 0], [40, 7, 300, 0, 64, 9, 1000], 2, 4, 64, 16)


def test_tokens_before_the_first_position_see_nothing():
    # more new tokens than the cache holds: the first ones stand before position 0
    _, _, out = run([5, 140], [2, 20], 1, 2, 64, 16)
    assert not out[:3].any() and not out[5:125].any()
    assert out[3:5].any() and out[125:].any()


def test_many_short_sequences():
    new = [(7 * i) % 5 for i in range(150)]
    run(new, [n + (i * 13) % 90 for i, n in enumerate(new)], 1, 2, 64, 16)


# Long prompts of many heads: several row tiles a sequence, several waves of them.

@pytest.mark.parametrize("dtype,codes", [("bf16", False), ("f16", False), ("bf16", True), ("f16", True)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_long_prompts(page, dtype, codes):
    # row tiles full, by one row more, of a pipe's rows alone, of few
    run([1100, 512, 513, 1700, 3, 0, 256], [1100, 2000, 513, 1701, 5, 40, 300], 26, 1, 128, page, dtype, codes)


@pytest.mark.parametrize("dim", [80, 96, 112])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("group", [3, 5])
def test_long_prompts_of_other_heads(group, codes, dim):
    run([399, 260, 129], [399, 1001, 640], 20, group, dim, 32, "bf16", codes, layout="tokens")


@pytest.mark.parametrize("window", [1, 100, 128, 700])
@pytest.mark.parametrize("codes", [False, True])
def test_long_prompts_in_a_window(window, codes):
    run([700, 600], [1500, 900], 32, 1, 128, 16, "bf16", codes, window=window)


@pytest.mark.parametrize("dtype,codes", [("bf16", False), ("f16", False), ("bf16", True), ("f16", True)])
def test_long_prompts_growing_maximum(dtype, codes):
    run([600, 650], [1500, 1300], 26, 1, 128, 16, dtype, codes, growth=6.0, q_scale=2.0)


def test_long_prompts_before_the_first_position():
    _, _, out = run([600, 700], [100, 660], 26, 1, 128, 16)
    assert not out[:500].any() and out[500:600].any() and not out[600:640].any() and out[640:].any()


# ------------------------------------------------------------------- masks --

@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 1000, 2 ** 40])
@pytest.mark.parametrize("codes", [False, True])
def test_window(window, codes):
    run([1, 150, 1], [700, 600, 50], 1, 4, 64, 16, "bf16", codes, window=window)


def test_pages_before_the_window_are_not_used():
    paged = Paged(torch, fw, 5, [1000], 1, 64, 16, "bf16", False, "heads")
    q = torch.randn((3, 4, 64), device=DEV).bfloat16()
    starts = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    a = fw.paged_attention(q, paged.cache, paged.table, paged.lens_t, starts=starts, window=100)
    paged.table[0, :(1000 - 3 - 100) // 16] = -1   # freed by a program that keeps the window only
    b = fw.paged_attention(q, paged.cache, paged.table, paged.lens_t, starts=starts, window=100)
    assert np.array_equal(bits(a), bits(b)) and fw.device_error() == 0


# -------------------------------------------------------------- softmax ----

@pytest.mark.parametrize("dtype,codes", [("bf16", False), ("f16", False), ("bf16", True), ("f16", True)])
def test_growing_maximum(dtype, codes):
    run([1, 90], [1500, 1300], 1, 4, 128, 16, dtype, codes, growth=6.0, q_scale=2.0)


def test_scale_argument_and_sharp_softmax():
    run([40], [500], 2, 4, 64, 16, "f16", scale=2.0)
    run([40], [500], 2, 4, 64, 16, "f16", scale=1e-3)


def test_equal_keys_give_the_mean():
    paged = Paged(torch, fw, 5, [384], 1, 64, 16, "f16", False, "heads")
    paged.cache.k.nan_to_num_(0.0).zero_()
    q = torch.randn((1, 2, 64), device=DEV).half()
    out = fw.paged_attention(q, paged.cache, paged.table, paged.lens_t)
    want = paged.rows[0][1][:, 0].mean(0).expand(1, 2, 64)
    assert float((out.double() - want).abs().max()) <= 2 ** -11 * float(want.abs().max()) + 384 * 2 ** -23 * 5


# --------------------------------------------------- calls and their order --

def test_same_bits_twice_on_another_stream_and_in_a_graph():
    q, paged, out = run([1, 80, 1], [3000, 500, 7], 2, 4, 128, 16)
    starts = torch.tensor([0, 1, 81, 82], dtype=torch.int32, device=DEV)
    first = bits(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = fw.paged_attention(q, paged.cache, paged.table, paged.lens_t, starts=starts)
    side.synchronize()
    assert np.array_equal(bits(again), first)
    held = torch.zeros_like(again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fw.paged_attention(q, paged.cache, paged.table, paged.lens_t, starts=starts, out=held)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(bits(held), first)


def test_pages_beyond_4_gib():
    # 40 pages 128 MiB apart: the last ones start past 2^32 bytes
    page, dim, stride = 16, 64, 1 << 26
    big = torch.empty(40 * stride, dtype=torch.bfloat16, device=DEV)
    k, v = (torch.as_strided(big, (40, 1, page, dim), (stride, page * dim, dim, 1), off) for off in (0, 1 << 20))
    for t in (k, v):
        t.copy_(torch.randn(t.shape, device=DEV))
    table = torch.arange(39, -1, -1, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([40 * page - 3], dtype=torch.int32, device=DEV)
    q = torch.randn((1, 4, dim), device=DEV).bfloat16()
    out = fw.paged_attention(q, fw.KVCache(k, v), table, lens)
    rows = [t.flip(0)[:, 0].reshape(-1, 1, dim)[:40 * page - 3].double() for t in (k, v)]
    want, tol = attend(torch, q.double(), rows[0], rows[1], 1, 40 * page - 3, dim ** -0.5, 0, "bf16")
    check(torch, out, want, tol)


def test_pages_beyond_4_gib_many_rows():
    page, dim, stride, n = 16, 128, 1 << 26, 30
    big = torch.empty(40 * stride, dtype=torch.bfloat16, device=DEV)
    k, v = (torch.as_strided(big, (40, 1, page, dim), (stride, page * dim, dim, 1), off) for off in (0, 1 << 20))
    for t in (k, v):
        t.copy_(torch.randn(t.shape, device=DEV))
    table = torch.arange(39, -1, -1, dtype=torch.int32, device=DEV)[None]
    length = 40 * page - 3
    lens, starts = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([length], [0, n]))
    q = torch.randn((n, 4, dim), device=DEV).bfloat16()
    out = fw.paged_attention(q, fw.KVCache(k, v), table, lens, starts=starts)
    rows = [t.flip(0)[:, 0].reshape(-1, 1, dim)[:length].double() for t in (k, v)]
    want, tol = attend(torch, q.double(), rows[0], rows[1], n, length, dim ** -0.5, 0, "bf16")
    check(torch, out, want, tol)


# ------------------------------------------------------ indices out of range

@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("entry", [-1, 10 ** 6, 2 ** 31 - 1])
def test_table_entry_outside_the_cache_is_recorded(entry, codes):
    paged = Paged(torch, fw, 5, [300, 300], 1, 64, 16, "bf16", codes, "heads")
    paged.table[1, 3] = entry
    q = torch.randn((2, 4, 64), device=DEV).bfloat16()
    out = fw.paged_attention(q, paged.cache, paged.table, paged.lens_t)
    assert fw.device_error() == 7006 and fw.device_error() == 0
    assert bool(torch.isfinite(out).all())
    want, tol = attend(torch, q[:1].double(), *paged.rows[0], 1, 300, 64 ** -0.5, 0, "bf16")
    check(torch, out[:1], want, tol)


def test_length_beyond_the_table_is_recorded():
    paged = Paged(torch, fw, 5, [300], 1, 64, 16, "bf16", False, "heads")
    q = torch.randn((1, 4, 64), device=DEV).bfloat16()
    for bad in (paged.table.shape[1] * 16 + 1, -1):
        out = fw.paged_attention(q, paged.cache, paged.table, torch.tensor([bad], dtype=torch.int32, device=DEV))
        assert fw.device_error() == 7006 and bool(torch.isfinite(out).all())


def test_starts_out_of_order_and_too_many_new_tokens_are_recorded():
    paged = Paged(torch, fw, 5, [300, 300], 1, 64, 16, "bf16", False, "heads")
    q = torch.randn((4, 4, 64), device=DEV).bfloat16()
    for starts in ([0, 3, 2], [0, 2, 5], [-1, 2, 4]):
        fw.paged_attention(q, paged.cache, paged.table, paged.lens_t, starts=torch.tensor(starts, dtype=torch.int32, device=DEV))
        assert fw.device_error() == 7006
    q = torch.randn((300, 4, 64), device=DEV).bfloat16()
    starts = torch.tensor([0, 299, 300], dtype=torch.int32, device=DEV)
    fw.paged_attention(q, paged.cache, paged.table, paged.lens_t, starts=starts, max_new=2)
    assert fw.device_error() == 7006
