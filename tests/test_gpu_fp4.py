"""GPU tests of the 4-bit form's weights: codes, blocks and scales bit for bit
what the rule gives in fp32 steps, values rounded once, and the linear layer
against the sum in 64 bits.

The bound of an output of the linear layer, with S = sum |x w| (64 bits) and u
the activation type's unit roundoff (2^-8 or 2^-11):
  u |y|                    the output rounded once (fp16: 2^-25 at least)
  + (k / 8 + 32) 2^-23 S   fp32 sums, each addition truncated at worst: a warp's
                           products add 16 terms a step, and the joins
  + 2^-38 max|x| sum|w|    (bf16) what a value loses below fp16's normal numbers
"""
import numpy as np
import pytest

from tests import fp4_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_weight_only_gb300 as fw  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def weights(seed, n, k):
    rng = np.random.default_rng(seed)
    w = rng.standard_normal((n, k)).astype(np.float32) * np.exp(rng.standard_normal((n, 1))).astype(np.float32)
    w[:, rng.integers(0, k, 3)] *= 20.0
    if n > 2:
        w[1] = 0.0                                  # a channel of zeros
        w[2, :16] = 0.0                             # a block of zeros
    return w


def same(got, want):
    assert np.array_equal(got.cpu().numpy().view(np.uint8), np.ascontiguousarray(want).view(np.uint8))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,k", [(1, 32), (9, 64), (5, 96), (33, 256), (300, 512), (7, 992), (4, 1024), (3, 1056), (5, 2048), (3, 4096),
                                 (2, 8224), (3, 14336), (2, 14368), (2, 28672), (2, 28704), (1, 65536)])
def test_quantize(n, k, dtype):
    w = torch.from_numpy(weights(k, n, k)).to(DT[dtype]).to(DEV)
    codes, blocks, scales = fw.quantize_fp4(w)
    want = R.quantize(w.float().cpu().numpy())
    same(codes, want[0])
    same(blocks, want[1])
    same(scales, want[2])


def test_quantize_of_the_ends_of_the_range():
    rng = np.random.default_rng(3)
    w = rng.standard_normal((8, 64)).astype(np.float32)
    w[0] *= np.float32(1e-42)                       # subnormal
    w[1] *= np.float32(1e-36)
    w[2] = np.abs(w[2]) * np.float32(1e38)
    w[3, 1:] = 0.0                                  # one value
    w[4] = -0.0
    w[5] = np.float32(6.0) * np.tile(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], np.float32) / 6, 8)  # the middles
    w[6, :16] *= np.float32(1e-5)                   # a block below the smallest scale of a block
    w[7] = 3.4e38
    got = fw.quantize_fp4(torch.from_numpy(w).to(DEV))
    for a, b in zip(got, R.quantize(w)):
        same(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,k", [(1, 32), (7, 96), (129, 992), (1000, 64), (3, 65536)])
def test_dequantize_rounds_once(n, k, dtype):
    codes, blocks, scales = R.quantize(weights(n + k, n, k))
    blocks[0, 0] = 1                                # the smallest block's scale
    want = R.values(codes, blocks, scales)
    buf = torch.full((n * k + 64,), 7.0, dtype=DT[dtype], device=DEV)
    t = [torch.from_numpy(a).to(DEV) for a in (codes, blocks, scales)]
    got = fw.dequantize_fp4(*t, out=buf[32:-32].view(n, k))
    assert bool((buf[:32] == 7).all()) and bool((buf[-32:] == 7).all())
    near = torch.from_numpy(want.astype(np.float32))           # 30 significant bits at most: one rounding for fp32
    if dtype == "f32":
        assert torch.equal(got.cpu(), near)
    else:
        d = (got.cpu().double() - torch.from_numpy(want)).abs()
        ulp = torch.from_numpy(want).abs() * U[dtype] + (2.0 ** -25 if dtype == "f16" else 0.0)
        assert bool((d <= ulp).all())
        rounded = torch.from_numpy(want).to(DT[dtype])         # torch rounds 64 bits through 32: ties aside the same
        assert float((got.cpu() != rounded).double().mean()) < 1e-3


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_dequantize_of_every_magnitude_rounds_once(dtype):
    """Scales from the smallest subnormal to the largest, against 64 bits rounded to
    the type's grid, its subnormal part too: a product has 30 bits, its quotient by
    the grid's step is exact in 64 bits, and rint takes ties to even."""
    rng = np.random.default_rng(17)
    n, k = 4096, 256
    codes, blocks = rng.integers(0, 256, (n, k // 2), dtype=np.uint8), rng.integers(0, 127, (n, k // 16), dtype=np.uint8)
    scales = np.ldexp(rng.integers(1, 1 << 24, n).astype(np.float64), rng.integers(-149, 93, n)).astype(np.float32)
    scales[:1024] = np.ldexp(rng.integers(1 << 23, (1 << 23) + 64, 1024).astype(np.float64), -149)  # at the smallest normal number
    scales[:4] = np.float32(2.0 ** -149), np.float32(2.0 ** -126), np.float32(2.0 ** -126 + 2.0 ** -149), np.float32(2.0 ** 112)
    scales[1::2] *= -1                              # a scale that is brought may be negative
    want = R.values(codes, blocks, scales)
    bits, lowest, most = {"f32": (24, -126, 128), "bf16": (8, -126, 128), "f16": (11, -14, 16)}[dtype]
    step = np.ldexp(1.0, np.maximum(np.frexp(want)[1] - 1, lowest) - (bits - 1))
    want = np.rint(want / step) * step
    want = np.where(np.abs(want) >= 2.0 ** most, np.copysign(np.inf, want), want)
    got = fw.dequantize_fp4(*(torch.from_numpy(a).to(DEV) for a in (codes, blocks, scales)), DT[dtype]).cpu().double().numpy()
    assert np.array_equal(got, want)


def test_dequantize_of_a_cache_shape():
    rng = np.random.default_rng(5)
    codes, blocks, scales = R.quantize(rng.standard_normal((3, 2, 16, 96)).astype(np.float32))
    t = [torch.from_numpy(a).to(DEV) for a in (codes, blocks, scales)]
    got = fw.dequantize_fp4(*t, torch.float32)
    assert torch.equal(got.cpu(), torch.from_numpy(R.values(codes, blocks, scales).astype(np.float32)))


def exact(x, codes, blocks, scales, bias):
    """(y, S, what bf16 may lose) in 64 bits on the GPU."""
    half = torch.from_numpy(R.E2M1).to(DEV)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    w = torch.cat([half, -half])[c] * torch.from_numpy(R.E4M3).to(DEV)[blocks.int()].repeat_interleave(16, -1) * scales.double()[:, None]
    xd = x.double()
    y = xd @ w.T
    if bias is not None:
        y = y + bias.double()
    s = xd.abs() @ w.abs().T + (0.0 if bias is None else bias.double().abs())
    lost = xd.abs().amax(1, keepdim=True) * w.abs().sum(1) * 2.0 ** -38
    return y, s, lost


def run(m, n, k, dtype="bf16", bias=True, seed=1, x=None, ready=False):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    if n * k < 10 ** 6:
        t = [torch.from_numpy(a).to(DEV) for a in R.quantize(weights(seed, n, k))]
    else:
        t = fw.quantize_fp4(torch.randn((n, k), generator=g, device=DEV))   # tested above
    if x is None:
        x = torch.randn((m, k), generator=g, device=DEV).to(DT[dtype])
    b = torch.randn(n, generator=g, device=DEV) if bias else None
    buf = torch.full((m * n + 64,), 7.0, dtype=DT[dtype], device=DEV)
    torch.cuda.synchronize()
    y = fw.linear_fp4(x, *t, b, out=buf[32:32 + m * n].view(m, n), weights_ready=ready)
    assert fw.device_error() == 0
    assert bool((buf[:32] == 7).all()) and bool((buf[-32:] == 7).all()), "written outside the output"
    want, s, lost = exact(x, *t, b)
    tol = U[dtype] * want.abs() + (k / 8 + 32) * 2.0 ** -23 * s + (lost if dtype == "bf16" else 2.0 ** -25)
    d = (y.double() - want).abs()
    assert bool(torch.isfinite(y).all())
    assert bool((d <= tol).all()), "off by up to %.3g of the bound" % float((d / tol).max())
    return y, x, t, b


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m", [1, 2, 3, 7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("n,k", [(1, 32), (17, 160), (130, 1024)])
def test_few_tokens(m, n, k, dtype):
    run(m, n, k, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m", [1, 5, 12, 29, 64])
@pytest.mark.parametrize("n,k", [(1000, 4096), (4096, 4128), (15, 14336), (20011, 96), (4100, 14336)])
def test_few_tokens_of_larger_layers(m, n, k, dtype):
    run(m, n, k, dtype, bias=m != 5, ready=m == 12)


@pytest.mark.parametrize("m", [1, 8, 9, 17, 33])
@pytest.mark.parametrize("n,k", [(40, 65536), (3000, 32800)])
def test_few_tokens_of_long_rows(m, n, k):
    run(m, n, k)


def test_joins_of_a_cluster_in_batches():
    # so many channels a cluster that their sums are joined several times
    run(32, 30000, 8192, "bf16", bias=False)
    run(7, 30001, 16384, "f16", bias=False)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m", [65, 128, 129, 300])
@pytest.mark.parametrize("n,k", [(1, 32), (127, 96), (130, 160), (256, 4096), (1001, 4128), (129, 224)])
def test_many_tokens(m, n, k, dtype):
    run(m, n, k, dtype, bias=n != 256, ready=n == 127)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(700, 2000, 4096), (257, 5000, 2080), (100, 20000, 1024), (129, 1000, 14336), (513, 300, 8192)])
def test_many_tokens_of_larger_layers(m, n, k, dtype):
    run(m, n, k, dtype)


@pytest.mark.parametrize("m", [3, 20, 90])
def test_activations_of_every_magnitude(m):
    # bf16 beyond fp16's range on both sides, in one token and between tokens
    g = torch.Generator(DEV)
    g.manual_seed(2)
    x = torch.randn((m, 256), generator=g, device=DEV)
    x *= torch.exp2(torch.randint(-10, 10, (m, 256), generator=g, device=DEV).float())
    x *= torch.exp2(torch.linspace(-100, 80, m, device=DEV))[:, None]
    x[0] = 0.0
    run(m, 48, 256, "bf16", bias=False, x=x.bfloat16())


@pytest.mark.parametrize("m", [2, 70])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_token_that_is_not_finite_changes_no_other(m, dtype):
    y, x, t, b = run(m, 40, 128, dtype)
    bad = x.clone()
    bad[1, 5], bad[1, 77] = float("inf"), float("nan")
    z = fw.linear_fp4(bad, *t, b)
    assert bool(torch.isnan(z[1]).all())
    keep = [i for i in range(m) if i != 1]
    assert torch.equal(z[keep], y[keep])


@pytest.mark.parametrize("m", [1, 6, 64, 100])
def test_results_are_the_same_every_time_and_in_a_graph(m):
    y, x, t, b = run(m, 1500, 4096)
    held = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        with torch.cuda.graph(held, stream=side):
            z = fw.linear_fp4(x, *t, b)
            z2 = fw.linear_fp4(x, *t, b, weights_ready=True)
    for _ in range(3):
        held.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, y) and torch.equal(z2, y)


def test_two_streams_at_once():
    y, x, t, b = run(5, 3000, 4096)
    y2, x2, t2, b2 = run(40, 2000, 2048, "f16", seed=2)
    a, c = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        with torch.cuda.stream(a):
            got.append((fw.linear_fp4(x, *t, b), y))
        with torch.cuda.stream(c):
            got.append((fw.linear_fp4(x2, *t2, b2), y2))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in got)


def test_a_layer_behind_the_quantiser_of_its_weight():
    """Quantise, multiply, and the next layer on the result, without a wait in between."""
    rng = np.random.default_rng(9)
    w = torch.from_numpy(rng.standard_normal((1024, 1024)).astype(np.float32)).to(DEV)
    x = torch.randn((3, 1024), device=DEV, dtype=torch.bfloat16)
    form = fw.quantize_fp4(w)
    torch.cuda.synchronize()
    one = fw.linear_fp4(x, *form)
    torch.cuda.synchronize()
    two = fw.linear_fp4(one, *form)
    torch.cuda.synchronize()
    for _ in range(5):
        f = fw.quantize_fp4(w)
        assert torch.equal(fw.linear_fp4(fw.linear_fp4(x, *f), *f), two)


def test_weights_past_four_gib():
    """Codes beyond 2^32 bytes: the last channels against those alone."""
    n, k, tail = 140000, 65536, 48
    g = torch.Generator(DEV)
    g.manual_seed(23)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    blocks = torch.randint(0x28, 0x48, (n, k // 16), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.rand((n,), generator=g, device=DEV) + 0.5
    ends = [t[-tail:].clone() for t in (codes, blocks, scales)]
    for m, dtype in ((1, "bf16"), (8, "f16"), (20, "bf16"), (100, "f16")):
        x = torch.randn((m, k), generator=g, device=DEV).to(DT[dtype])
        y = fw.linear_fp4(x, codes, blocks, scales)[:, -tail:]
        want, total, lost = exact(x, *ends, None)
        tol = U[dtype] * want.abs() + (k / 8 + 32) * 2.0 ** -23 * total + (lost if dtype == "bf16" else 2.0 ** -25)
        assert bool(((y.double() - want).abs() <= tol).all())
    assert fw.device_error() == 0
    w = fw.dequantize_fp4(codes, blocks, scales)
    want = fw.dequantize_fp4(*ends)
    assert torch.equal(w[-tail:], want)
    del codes, blocks
    for got, alone in zip(fw.quantize_fp4(w), fw.quantize_fp4(want)):
        assert torch.equal(got[-tail:], alone)


def test_the_binding_checks_its_operands():
    codes, blocks, scales = fw.quantize_fp4(torch.randn((8, 64), device=DEV))
    x = torch.randn((2, 64), device=DEV).bfloat16()
    for bad in ((x.float(), codes, blocks, scales), (x[:, ::2], codes, blocks, scales), (x, codes.int(), blocks, scales),
                (x, codes, blocks, scales.double()), (x.cpu(), codes, blocks, scales), (x, codes.cpu(), blocks, scales)):
        with pytest.raises(TypeError):
            fw.linear_fp4(*bad)
    for bad in ((x, codes[:, :16], blocks, scales), (x, codes, blocks[:4], scales), (x, codes, blocks, scales[:3])):
        with pytest.raises((TypeError, ValueError)):
            fw.linear_fp4(*bad)
    with pytest.raises((TypeError, ValueError)):
        fw.linear_fp4(x, codes, blocks, scales, torch.zeros(7, device=DEV))
    with pytest.raises(ValueError):
        fw.linear_fp4(x, codes, blocks, scales, out=torch.empty((2, 7), device=DEV, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        fw.quantize_fp4(torch.zeros((4, 64), device=DEV, dtype=torch.int32))
    with pytest.raises(fw.Fp8wError):
        fw.quantize_fp4(torch.zeros((4, 48), device=DEV))
    with pytest.raises(TypeError):
        fw.quantize_fp4(torch.zeros((4, 64), device=DEV), codes=torch.zeros((4, 64), dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        fw.dequantize_fp4(codes, blocks[:, :2].contiguous(), scales)
    with pytest.raises(TypeError):
        fw.dequantize_fp4(codes, blocks, scales, torch.int32)
