"""The example's attention block (FP8 projections, rotary positions, append,
paged attention, chunked prompts, decoding from a CUDA graph) against the same
block in 64 bits without any of its roundings.

Tolerance, relative L2 of a token's output.  A 16-bit rounding is off by
2^-8 / sqrt(12) of the value's power of two, at most 2^-8 / sqrt(12) = 1.1e-3
of the value itself.  The value projection, the softmax weights, the
attention's result and the output have one each; queries and keys two each,
which move a score of about unit size by 2 * 1.1e-3 and its weight as much,
as two values of a sum of independent ones: sqrt(4 * 1.1^2 + 2 * 2.2^2) e-3
= 3.8e-3 in all; 2^-7 is twice that.  Codes add e4m3's 2^-3 / sqrt(12) = 3.6e-2
at the worst place of a power of two to values and, through the scores, to
weights: 5.1e-2; the bound is 2^-3."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_weight_only_gb300 as fw  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import attention_block as ex  # noqa: E402


def plain(block, x):
    """All tokens of one sequence at once, 64 bits, causal."""
    def product(t, weights):
        codes, scales = weights
        return t @ (codes.view(torch.float8_e4m3fn).double() * scales.double()[:, None]).T

    n, d = len(x), block.head_dim
    qkv = product(x.double(), block.qkv).view(n, -1, d)
    q, k, v = qkv.split([block.heads, block.kv_heads, block.kv_heads], 1)
    cos, sin = block.rope.table[:n].double().chunk(2, 1)

    def turned(t):
        a, b = t.chunk(2, -1)
        return torch.cat([a * cos[:, None] - b * sin[:, None], b * cos[:, None] + a * sin[:, None]], -1)

    group = block.heads // block.kv_heads
    q, k, v = turned(q), turned(k).repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    s = torch.einsum("qhd,khd->hqk", q, k) * d ** -0.5
    s = s.masked_fill(torch.ones((n, n), dtype=torch.bool, device=x.device).triu(1), -float("inf"))
    return product(torch.einsum("hqk,khd->qhd", s.softmax(-1), v).reshape(n, -1), block.o)


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("heads,kv_heads,head_dim,page,prompts", [(8, 2, 64, 16, (300, 1, 129)), (12, 4, 128, 64, (65, 257))])
def test_block(heads, kv_heads, head_dim, page, prompts, codes):
    steps = 5
    block, pages, x = ex.build(heads, kv_heads, head_dim, 512, page, prompts, steps, codes)
    got = ex.prefill(block, pages, [t[:n] for t, n in zip(x, prompts)], 128)
    decode = ex.Decoder(block, pages, 512)
    for i in range(steps):
        y = decode(torch.stack([t[n + i] for t, n in zip(x, prompts)]))
        got = [torch.cat([g, y[b:b + 1]]) for b, g in enumerate(got)]
    assert fw.device_error() == 0
    for b, t in enumerate(x):
        want = plain(block, t)
        off = (got[b].double() - want).norm(dim=1) / want.norm(dim=1)
        assert float(off.max()) <= (2.0 ** -3 if codes else 2.0 ** -7), "token %d off by %.3g" % (int(off.argmax()), float(off.max()))
