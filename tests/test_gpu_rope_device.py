"""GPU test: a table on another device than the operands is refused.  (One GPU:
the device that the Rope notes of its table is changed instead.)"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_weight_only_gb300 as fw  # noqa: E402

DEV = torch.device("cuda:0")


def test_a_table_on_another_device_is_refused():
    spec = fw.Rope(torch.zeros((8, 64), device=DEV))
    x = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device=DEV)
    pos, slots = torch.zeros(2, dtype=torch.int32, device=DEV), torch.arange(2, device=DEV)
    pages = torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16, device=DEV)
    cache = fw.KVCache(pages, pages.clone())
    assert spec.index == DEV.index
    fw.rope(x, pos, spec)
    fw.rope_append(x, x, x, slots, cache, pos, spec)
    spec.index += 1
    with pytest.raises(TypeError, match="device"):
        fw.rope(x, pos, spec)
    with pytest.raises(TypeError, match="device"):
        fw.rope_append(x, x, x, slots, cache, pos, spec)
