"""dequantize_fp4 of scales and blocks that are not finite: what the product is."""
import numpy as np
import pytest

from tests import fp4_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_weight_only_gb300 as fw  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_products_that_are_not_finite(dtype):
    rng = np.random.default_rng(4)
    n, k = 6, 96
    codes, blocks = rng.integers(0, 256, (n, k // 2), dtype=np.uint8), rng.integers(1, 127, (n, k // 16), dtype=np.uint8)
    codes[:, 0] = 0x08                              # zeros of both signs: times infinity NaN
    blocks[:, 2] = 0
    blocks[3, 3] = 0x7F                             # a block of NaN
    scales = np.array([np.inf, -np.inf, np.nan, 1.5, 3.0e38, 0.0], np.float32)
    with np.errstate(invalid="ignore"):
        want = R.values(codes, blocks, scales)
    got = fw.dequantize_fp4(*(torch.from_numpy(a).to("cuda") for a in (codes, blocks, scales)), dtype).cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(want).any()
    most = float(torch.finfo(dtype).max) * (1 + torch.finfo(dtype).eps / 4)   # beyond: infinite
    huge = np.abs(want) >= most
    assert huge.any() and np.array_equal(got[huge], np.copysign(np.inf, want[huge]))
    assert np.isfinite(got[~huge & ~np.isnan(want)]).all()
