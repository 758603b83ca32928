"""GPU tests of fp8w_paged_attention where the softmax weights reach far down: a
few dominant keys over a long tail, small values, values whose size differs
from token to token and head to head, keys of the largest scores whose values
are zero.

Weights that are held in fp16 are off by 2^-11 of themselves or, below its
normal range, by 2^-25 of a unit of which the largest weight (with codes:
weight times value) has at least 2^7: by 2^-32 of that one.  So the bound is
that of attention_reference with the term for weights below the normal range
replaced by  keys 2^-32 max_j p_j max_d |v_jd|  (with 16-bit pages, where it is
the weight alone that is held: keys 2^-32 max_j p_j max |v|).  The bound shrinks
with the values.  fp16 outputs below its normal range are off by 2^-25."""
import pytest

from tests.attention_reference import ROUND, check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_weight_only_gb300 as fw  # noqa: E402

DEV = torch.device("cuda:0")


def paged(k, v, page, dtype, codes):
    """A cache that holds k and v [length, kv_heads, dim] in shuffled pages:
    (cache, table, the held k and v in 64 bits)."""
    length, kv, dim = k.shape
    pages = -(-length // page)
    table = torch.randperm(pages, device=DEV).int()[None]
    held, parts = [], []
    for x in (k, v):
        padded = torch.zeros((pages * page, kv, dim), device=DEV)
        padded[:length] = x
        scales = None
        if codes:
            scales = padded.abs().amax(-1) / 448.0
            scales[scales == 0] = 1.0
            q = (padded / scales[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            held.append(q[:length].double() * scales[:length, :, None].double())
            padded = q.view(torch.uint8)
        else:
            padded = padded.to(torch.bfloat16 if dtype == "bf16" else torch.float16)
            held.append(padded[:length].double())
        for t in (padded, scales):
            if t is not None:
                rows = t.view(pages, page, *t.shape[1:]).transpose(1, 2)
                t = torch.empty_like(rows, memory_format=torch.contiguous_format)
                t[table[0].long()] = rows
            parts.append(t)
    return fw.KVCache(parts[0], parts[2], parts[1], parts[3]), table, held


def compare(k, v, new, group, dtype, codes, page=32):
    """Queries 4 e_0, scale 1: key j's score is 4 k_j0.  Returns the largest
    share of the bound that was used."""
    length, kv, dim = k.shape
    cache, table, (hk, hv) = paged(k, v, page, dtype, codes)
    q = torch.zeros((new, kv * group, dim), dtype=torch.bfloat16 if dtype == "bf16" else torch.float16, device=DEV)
    q[..., 0] = 4.0
    lens, starts = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([length], [0, new]))
    out = fw.paged_attention(q, cache, table, lens, starts=starts, scale=1.0, max_new=new, max_len=length)
    assert fw.device_error() == 0
    seen = torch.arange(length, device=DEV) <= length - new + torch.arange(new, device=DEV)[:, None]
    u, want, tol = ROUND[dtype], torch.empty(q.shape, dtype=torch.float64, device=DEV), torch.empty(q.shape, dtype=torch.float64, device=DEV)
    for h in range(kv):
        s = torch.where(seen, 4.0 * hk[:, h, 0], -float("inf"))
        p = torch.softmax(s, -1)
        o, a = p @ hv[:, h], p @ hv[:, h].abs()
        big = (p * hv[:, h].abs().amax(-1)).amax(-1) if codes else p.amax(-1) * hv[:, h].abs().max()
        e_s = (dim + 8) * 2.0 ** -23 * 4.0 * hk[:, h, 0].abs().max() + 2.0 ** -18
        t = u * (a + o.abs()) + 2 * e_s * a + length * 2.0 ** -23 * a
        if dtype == "f16" or codes:
            t = t + length * 2.0 ** -32 * big[:, None]
        if dtype == "f16":
            t = t + 2.0 ** -25
        for g in range(group):
            want[:, h * group + g], tol[:, h * group + g] = o, t
    return check(torch, out, want, tol)


def tail(length, kv, dim, down, seed=2):
    """Keys whose scores lie `down` to down + 1 below those of three dominant
    ones, and values in [0.5, 1] with a 1 in each row."""
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    k = torch.zeros((length, kv, dim), device=DEV)
    k[..., 0] = -(down + torch.rand((length, kv), generator=g, device=DEV)) / 4.0
    for at in (7, length // 2, length // 3):
        k[at, :, 0] = 0.0
    v = 0.5 + 0.5 * torch.rand((length, kv, dim), generator=g, device=DEV)
    v[..., dim // 2] = 1.0
    return k, v


# new tokens and query heads a key head: few rows, few rows of two tiles of 8, a tile of many, a tile a pipe
ROWS = [(1, 4), (3, 5), (60, 1), (200, 2)]
FORMS = [("bf16", False), ("f16", False), ("bf16", True), ("f16", True)]


@pytest.mark.parametrize("new,group", ROWS)
@pytest.mark.parametrize("dtype,codes", FORMS)
@pytest.mark.parametrize("amax", [3.0, 0.1, 0.01, 0.001])
def test_small_values_under_a_long_tail(amax, dtype, codes, new, group):
    k, v = tail(9000, 2, 64, 9.0)
    compare(k, v * amax, new, group, dtype, codes)


@pytest.mark.parametrize("new,group", ROWS)
@pytest.mark.parametrize("dtype,codes", FORMS)
@pytest.mark.parametrize("dim", [64, 128])
def test_values_of_mixed_size(dim, dtype, codes, new, group):
    k, v = tail(5000, 2, dim, 7.0)
    g = torch.Generator(DEV)
    g.manual_seed(8)
    compare(k, v * 10.0 ** (-4.0 * torch.rand((5000, 2, 1), generator=g, device=DEV)), new, group, dtype, codes)


@pytest.mark.parametrize("new,group", ROWS)
@pytest.mark.parametrize("dtype,codes", FORMS)
@pytest.mark.parametrize("amax", [1.0, 0.1, 0.001])
@pytest.mark.parametrize("dim", [64, 128])
def test_keys_of_the_largest_scores_with_zero_values(dim, amax, dtype, codes, new, group):
    # padded or null tokens at the start, in the middle and among the last
    k, v = tail(3000, 2, dim, 9.0)
    for at in (0, 7, 1500, 1000, 2790):
        k[at, :, 0], v[at] = 0.5, 0.0
    compare(k, v * amax, new, group, dtype, codes)


@pytest.mark.parametrize("new,group", ROWS)
@pytest.mark.parametrize("dtype,codes", FORMS)
def test_all_values_zero(dtype, codes, new, group):
    k, v = tail(300, 2, 64, 9.0)
    assert compare(k, v * 0.0, new, group, dtype, codes) == 0.0


@pytest.mark.parametrize("new,group", ROWS)
@pytest.mark.parametrize("codes", [False, True])
def test_value_scale_of_exactly_one(codes, new, group):
    # 448 is the value whose row has the scale of a row of zeros
    k, v = tail(3000, 2, 64, 9.0)
    v = torch.where(v == 1.0, 448.0, v)
    v[::3] *= 1e-3
    compare(k, v, new, group, "f16", codes)


@pytest.mark.parametrize("new,group", ROWS)
@pytest.mark.parametrize("codes", [False, True])
def test_weights_below_2_to_the_minus_25(codes, new, group):
    # the dominant keys, one in 16, have zero values: what the output has comes from the others
    k, v = tail(512, 2, 64, 17.6)
    k[7::16, :, 0], v[7::16], v[256], v[170] = 0.0, 0.0, 0.0, 0.0
    compare(k, v * 2.0 ** 15, new, group, "f16", codes)


def test_bf16_values_of_extreme_size():
    # scales from 2^-100 on, where a weight times its scale is a normal fp16 number only by the reference
    k, v = tail(2000, 2, 64, 5.0)
    for size in (2.0 ** -90, 2.0 ** 100):
        for new, group in ROWS:
            compare(k, v * size, new, group, "bf16", True)
