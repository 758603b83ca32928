"""The 4-bit linear layer where the rings of its tensor-core kernels go round often:
several tiles a CTA of any number of k-blocks, and weights that are ready long before
the activations are, so that the dequantising warps are as far ahead as the rings let
them.  Bounds as in test_gpu_fp4.py; and the same bits every time, with the weights
waited for and without.  (What the rings rely on: test_rings.py.)"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_weight_only_gb300 as fw  # noqa: E402
from tests.test_gpu_fp4 import DEV, DT, U, exact, run  # noqa: E402


def behind_a_long_kernel(m, n, k, dtype, seed=3):
    """x comes from a kernel of few CTAs that runs for long."""
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    long_k = 65536
    first = fw.quantize(torch.randn((k, long_k), generator=g, device=DEV) * long_k ** -0.5)
    form = fw.quantize_fp4(torch.randn((n, k), generator=g, device=DEV))
    x0 = torch.randn((m, long_k), generator=g, device=DEV).to(DT[dtype])
    flush = torch.empty(160 << 20, dtype=torch.uint8, device=DEV)
    x = fw.linear(x0, *first)
    torch.cuda.synchronize()
    y = fw.linear_fp4(x, *form)
    torch.cuda.synchronize()
    want, s, lost = exact(x, *form, None)
    tol = U[dtype] * want.abs() + (k / 8 + 32) * 2.0 ** -23 * s + (lost if dtype == "bf16" else 2.0 ** -25)
    assert bool(((y.double() - want).abs() <= tol).all())
    z = torch.empty_like(x)
    out = torch.empty_like(y)
    for ready in (True, False, True, True):
        z.fill_(float("nan"))
        out.fill_(float("nan"))
        flush.fill_(1)                    # weights and blocks' scales out of L2
        torch.cuda.synchronize()
        fw.linear(x0, *first, out=z)
        fw.linear_fp4(z, *form, out=out, weights_ready=ready)
        torch.cuda.synchronize()
        assert torch.equal(z, x) and torch.equal(out, y)
    assert fw.device_error() == 0


# 2 or 3 tiles for each SM, and so few k-blocks that the prefill GEMM takes them
PROMPTS = [(65, 40009, b) for b in (5, 6, 7, 14, 18)] + [(300, 20011, b) for b in (5, 6, 7, 14, 18, 45, 67)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,blocks", PROMPTS)
def test_prompts_of_several_tiles_of_any_k_blocks(m, n, blocks, dtype):
    k = 64 * blocks - (32 if m == 300 else 0)
    y, x, t, b = run(m, n, k, dtype)
    for _ in range(4):
        assert torch.equal(fw.linear_fp4(x, *t, b, weights_ready=True), y)
    assert fw.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,blocks", PROMPTS)
def test_prompts_behind_a_long_kernel(m, n, blocks, dtype):
    behind_a_long_kernel(m, n, 64 * blocks, dtype)


# clusters that share a tile, tiles of an SM's own, rows that end inside a unit; prompts
# that go by slabs of 64 tokens
FEW = [(16, 14336, 4096), (9, 40009, 1152), (32, 10007, 4128), (23, 4100, 14336), (64, 14336, 4096), (40, 30011, 2080), (65, 40009, 2880),
       (65, 40009, 4288)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", FEW)
def test_tokens_of_many_units(m, n, k, dtype):
    y, x, t, b = run(m, n, k, dtype)
    for _ in range(20):
        assert torch.equal(fw.linear_fp4(x, *t, b), y)
    assert fw.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", FEW)
def test_tokens_behind_a_long_kernel(m, n, k, dtype):
    behind_a_long_kernel(m, n, k, dtype)
