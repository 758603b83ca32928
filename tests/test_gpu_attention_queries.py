"""GPU tests of fp8w_paged_attention with queries that are not finite: by the
definition the whole row is NaN (a NaN score, or an infinite one less itself),
in every form of the kernels, and the other rows keep their bits.  A row that
sees nothing is zeros whatever its query."""
import numpy as np
import pytest

from tests.attention_reference import Paged, bits

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_weight_only_gb300 as fw  # noqa: E402

DEV = torch.device("cuda:0")

FORMS = [
    # new tokens, lengths, query heads a key head, head size, max_new
    ([1, 1], [1, 300], 4, 128, 1),        # few rows, a CTA a sequence
    ([1], [9000], 8, 64, 1),              # few rows, split over a cluster
    ([4, 3], [700, 20], 4, 128, 4),       # few rows, two tiles of 8 a product
    ([12, 1], [5000, 40], 4, 64, 12),     # few rows with codes, several tiles over a cluster; else one tile of many
    ([64, 1], [64, 500], 1, 128, 64),     # many rows: both pipes on one tile's rows
    ([20], [600], 5, 64, 0),              # many rows, fewer than a tile
    ([300], [300], 2, 128, 0),            # a tile a pipe, written without a join
    ([64], [6000], 4, 128, 0),            # a tile a pipe over a cluster
    ([50], [9000], 1, 64, 0),             # a tile over a cluster
]


@pytest.mark.parametrize("dtype,codes", [("bf16", False), ("f16", False), ("bf16", True), ("f16", True)])
@pytest.mark.parametrize("new,lens,group,dim,max_new", FORMS)
def test_a_query_that_is_not_finite_makes_its_row_nan(new, lens, group, dim, max_new, dtype, codes):
    paged = Paged(torch, fw, 9, lens, 2, dim, 16, dtype, codes, "heads")
    tokens, heads = sum(new), 2 * group
    g = torch.Generator(DEV)
    g.manual_seed(3)
    clean = torch.randn((tokens, heads, dim), generator=g, device=DEV).to(torch.bfloat16 if dtype == "bf16" else torch.float16)
    starts = torch.tensor([0] + new, device=DEV).cumsum(0).int()

    def run(q):
        out = fw.paged_attention(q, paged.cache, paged.table, paged.lens_t, starts=starts, max_new=max_new)
        assert fw.device_error() == 0
        return out

    want = run(clean)
    bad = clean.clone()
    rows = [(0, heads - 1, float("nan"), 5), (tokens - 1, 0, float("inf"), dim - 1), (tokens // 2, heads // 2, -float("inf"), 0)]
    hit = torch.zeros((tokens, heads), dtype=torch.bool, device=DEV)
    for t, h, x, d in rows:
        bad[t, h, d] = x
        hit[t, h] = True
    got = run(bad)
    assert bool(torch.isnan(got[hit]).all())
    assert np.array_equal(bits(got[~hit]), bits(want[~hit]))


@pytest.mark.parametrize("dtype,codes", [("bf16", False), ("f16", True)])
@pytest.mark.parametrize("group", [1, 100])
def test_scores_of_minus_infinity_alone(group, dtype, codes):
    # one key that points away from an infinite query: exp(-inf - -inf)
    paged = Paged(torch, fw, 9, [1], 1, 64, 16, dtype, codes, "heads")
    q = torch.zeros((1, group, 64), dtype=torch.bfloat16 if dtype == "bf16" else torch.float16, device=DEV)
    key = paged.rows[0][0][0, 0]
    q[0, 0] = torch.where(key > 0, -float("inf"), float("inf")).to(q.dtype)
    q[0, 0, key == 0] = 0
    out = fw.paged_attention(q, paged.cache, paged.table, paged.lens_t)
    assert bool(torch.isnan(out[0, 0]).all())
    if group > 1:
        assert bool((out[0, 1:].double() - paged.rows[0][1][0, 0]).abs().max() <= 2.0 ** -7 * paged.rows[0][1].abs().max())


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("new", [1, 200])
def test_a_row_that_sees_nothing_is_zero_whatever_its_query(new, codes):
    paged = Paged(torch, fw, 9, [0], 1, 64, 16, "bf16", codes, "heads")
    q = torch.full((new, 2, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    starts = torch.tensor([0, new], dtype=torch.int32, device=DEV)
    assert not fw.paged_attention(q, paged.cache, paged.table, paged.lens_t, starts=starts).any()
