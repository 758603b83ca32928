"""GPU tests of the forms of paged attention that a call with max_new reaches:
few rows in tiles of 16, one tile and several a sequence, with 16-bit pages and
codes, windows and splits over a cluster; hints beyond all bounds."""
import numpy as np
import pytest

from tests.attention_reference import Paged, bits
from tests.test_gpu_attention import run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_weight_only_gb300 as fw  # noqa: E402

DEV = torch.device("cuda:0")
FORMS = [("bf16", False), ("f16", False), ("bf16", True), ("f16", True)]


@pytest.mark.parametrize("dtype,codes", FORMS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,group", [(3, 3), (4, 4), (17, 1), (11, 3), (12, 4), (3, 16)])   # 9, 16, 17, 33, 48, 48 rows
def test_few_rows_in_tiles_of_sixteen(new, group, dim, dtype, codes):
    run([new, 1, 0, new - 1], [400, 70, 9, 33], 2, group, dim, 16, dtype, codes, max_new=new)


@pytest.mark.parametrize("dtype,codes", FORMS)
@pytest.mark.parametrize("dim", [48, 80, 112])
def test_few_rows_of_other_heads(dim, dtype, codes):
    run([3, 4], [130, 70], 2, 4, dim, 32, dtype, codes, layout="tokens", max_new=4)


@pytest.mark.parametrize("dtype,codes", FORMS)
@pytest.mark.parametrize("dim", [64, 128])
def test_few_rows_in_a_window(dim, dtype, codes):
    run([4, 2, 4], [700, 50, 4], 2, 4, dim, 16, dtype, codes, window=100, max_new=4)
    if codes:
        run([12, 12], [700, 12], 2, 4, dim, 16, dtype, codes, window=5, max_new=12)


@pytest.mark.parametrize("dtype,codes", FORMS)
@pytest.mark.parametrize("dim", [64, 128])
def test_few_rows_split_over_a_cluster(dim, dtype, codes):
    run([4], [6001], 1, 4, dim, 64, dtype, codes, max_new=4, growth=4.0)
    if codes:
        run([12, 5], [6001, 3000], 1, 4, dim, 64, dtype, codes, max_new=12, growth=4.0)


@pytest.mark.parametrize("dtype,codes", FORMS)
def test_few_rows_before_the_first_position(dtype, codes):
    _, _, out = run([4, 4], [2, 0], 2, 4, 64, 16, dtype, codes, max_new=4)
    assert not out[:2].any() and out[2:4].any() and not out[4:].any()


@pytest.mark.parametrize("dtype,codes", FORMS)
@pytest.mark.parametrize("dim", [64, 128])
def test_a_tile_of_rows_before_the_first_position_beside_one_that_sees_keys(dim, dtype, codes):
    # 128 rows that see nothing and 128 of which the last do, many times over: the first
    # ones' zeros are written while the queries may still be on their way
    new, lens = [256] * 40, [12 + i for i in range(40)]
    for seed in range(20):
        _, _, out = run(new, lens, 8, 1, dim, 16, dtype, codes, seed=seed)
        for b, t in enumerate(lens):
            assert not out[256 * b:256 * (b + 1) - t].any()


@pytest.mark.parametrize("max_new", [2 ** 62, 2 ** 62 + 1, 2 ** 63 - 1])
def test_a_bound_on_new_tokens_above_all_tokens_is_no_bound(max_new):
    for new, lens in (([1, 3], [700, 90]), ([200, 7], [300, 90])):
        _, _, want = run(new, lens, 2, 4, 64, 16)
        _, _, got = run(new, lens, 2, 4, 64, 16, max_new=max_new)
        assert np.array_equal(bits(got), bits(want))


@pytest.mark.parametrize("new,lens", [([1, 1], [9000, 0]), ([3, 5], [700, 2]), ([200, 300], [9000, 20])])
def test_a_window_above_all_positions_is_none(new, lens):
    paged = Paged(torch, fw, 5, lens, 1, 64, 16, "bf16", False, "heads")
    q = torch.randn((sum(new), 4, 64), device=DEV).bfloat16()
    starts = torch.tensor([0] + new, device=DEV).cumsum(0).int()
    want = fw.paged_attention(q, paged.cache, paged.table, paged.lens_t, starts=starts)
    for window in (9100, 2 ** 31, 2 ** 62, 2 ** 63 - 1):
        got = fw.paged_attention(q, paged.cache, paged.table, paged.lens_t, starts=starts, window=window)
        assert np.array_equal(bits(got), bits(want))
    assert fw.device_error() == 0


@pytest.mark.parametrize("dtype,codes", FORMS)
@pytest.mark.parametrize("dim", [16, 32, 48])
def test_many_rows_of_small_heads(dim, dtype, codes):
    run([300, 20], [300, 700], 2, 3, dim, 16, dtype, codes)
    run([64], [5000], 1, 1, dim, 128, dtype, codes, layout="tokens")
