"""GPU test of appends and attentions one behind the other in the stream: each
starts while those ahead of it still run, and gives what it gives when the
device is waited for in between."""
import pytest

from tests.attention_reference import bits

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_weight_only_gb300 as fw  # noqa: E402

DEV = torch.device("cuda:0")


def chain(codes, group, seqs, steps, graph):
    """The outputs of `steps` new tokens of each sequence, one at a time: each
    step writes a slot beside those it wrote before, in the same pages."""
    kv, dim, page, width = 2, 128, 16, 8
    g = torch.Generator(DEV)
    g.manual_seed(4)
    dtype = torch.uint8 if codes else torch.bfloat16
    k, v = (torch.zeros((seqs * width, kv, page, dim), dtype=dtype, device=DEV) for _ in range(2))
    ks, vs = (torch.ones(k.shape[:3], device=DEV) if codes else None for _ in range(2))
    cache = fw.KVCache(k, v, ks, vs)
    table = torch.randperm(seqs * width, generator=g, device=DEV).int().view(seqs, width)
    fused = torch.randn((steps, seqs, kv * (group + 2), dim), generator=g, device=DEV).bfloat16()
    angle = torch.arange(steps, device=DEV)[:, None] * 100.0 ** -torch.linspace(0, 1, dim // 2, device=DEV)
    rope = fw.Rope(torch.cat([angle.cos(), angle.sin()], 1).contiguous())
    at = torch.arange(steps, device=DEV)
    slots = (table.long()[:, at // page] * page + at % page).t().contiguous()
    lens = (at[:, None] + 1).int().expand(steps, seqs).contiguous()
    positions = at[:, None].int().expand(steps, seqs).contiguous()

    def run(wait):
        outs = []
        for i in range(steps):
            q, key, value = fused[i].split([kv * group, kv, kv], 1)
            q = fw.rope_append(q, key, value, slots[i], cache, positions[i], rope)
            if wait:
                torch.cuda.synchronize()
            outs.append(fw.paged_attention(q, cache, table, lens[i]))
            if wait:
                torch.cuda.synchronize()
        return torch.stack(outs)

    if not graph:
        return run(True)
    held = torch.cuda.CUDAGraph()
    with torch.cuda.graph(held):
        out = run(False)
    held.replay()
    torch.cuda.synchronize()
    return out.clone()   # the graph's memory goes with it


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("group,seqs", [(4, 1), (4, 150), (60, 3)])   # few rows: one cluster, many CTAs; many rows
def test_calls_in_a_row_give_what_calls_apart_give(group, seqs, codes):
    steps = 100
    assert (bits(chain(codes, group, seqs, steps, False)) == bits(chain(codes, group, seqs, steps, True))).all()
    assert fw.device_error() == 0
