"""The attention half of a decoder block, as a server runs it: FP8 q/k/v
projection, rotary positions, a paged cache, attention over it, FP8 output
projection.

    python examples/attention_block.py [--codes] [--steps N]

A block of 32 query and 8 key heads of 128 takes three prompts of different
lengths in chunks, then decodes a token of each at a time; the decoding step is
captured once in a CUDA graph and replayed.  The cache holds bf16 values, or
with --codes e4m3 codes and a scale a slot and head.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_weight_only_gb300 as fw  # noqa: E402


def rope_table(max_pos, rot_dim, base=10000.0, device="cuda"):
    """[max_pos, rot_dim]: cosines, then sines, of pos * base^(-2 i / rot_dim)."""
    rates = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    angles = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * rates
    return torch.cat([angles.cos(), angles.sin()], 1).float().contiguous()


class Pages:
    """A paged cache and the host's book of who owns which page."""

    def __init__(self, num_pages, page_size, kv_heads, head_dim, seqs, width, codes, device="cuda"):
        shape = (num_pages, kv_heads, page_size, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8 if codes else torch.bfloat16, device=device) for _ in range(2))
        ks, vs = (torch.zeros(shape[:3], device=device) if codes else None for _ in range(2))
        self.cache = fw.KVCache(k, v, ks, vs)
        self.page_size, self.free = page_size, list(range(num_pages))[::-1]
        self.owned = [[] for _ in range(seqs)]
        self.lens = [0] * seqs
        self.table = torch.full((seqs, width), -1, dtype=torch.int32)

    def grow(self, seq, tokens):
        """Room for `tokens` more of a sequence; their positions and slots."""
        positions = list(range(self.lens[seq], self.lens[seq] + tokens))
        self.lens[seq] += tokens
        while len(self.owned[seq]) * self.page_size < self.lens[seq]:
            page = self.free.pop()
            self.table[seq, len(self.owned[seq])] = page
            self.owned[seq].append(page)
        slots = [self.owned[seq][p // self.page_size] * self.page_size + p % self.page_size for p in positions]
        return positions, slots


class AttentionBlock:
    """y = attention(x Wqkv^T) Wo^T; weights e4m3 with a scale a row."""

    def __init__(self, wqkv, wo, heads, kv_heads, head_dim, rope):
        self.qkv, self.o = fw.quantize(wqkv), fw.quantize(wo)
        self.heads, self.kv_heads, self.head_dim, self.rope = heads, kv_heads, head_dim, rope

    def __call__(self, x, positions, slots, cache, table, lens, starts=None, max_new=0, max_len=0):
        qkv = fw.linear(x, *self.qkv, weights_ready=True)
        # views of the fused rows: the kernels take the rows' stride
        q, k, v = qkv.view(len(x), -1, self.head_dim).split([self.heads, self.kv_heads, self.kv_heads], 1)
        q = fw.rope_append(q, k, v, slots, cache, positions, self.rope)
        out = fw.paged_attention(q, cache, table, lens, starts=starts, max_new=max_new, max_len=max_len)
        return fw.linear(out.view(len(x), -1), *self.o, weights_ready=True)


def device_int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def prefill(block, pages, prompts, chunk):
    """Prompts [tokens, hidden] in chunks of all sequences together; outputs of each."""
    outs = [[] for _ in prompts]
    for first in range(0, max(len(p) for p in prompts), chunk):
        parts = [p[first:first + chunk] for p in prompts]
        new = [len(p) for p in parts]
        placed = [pages.grow(b, n) for b, n in enumerate(new)]
        starts = [sum(new[:b]) for b in range(len(new) + 1)]
        y = block(torch.cat(parts), device_int([p for at in placed for p in at[0]]),
                  device_int([s for at in placed for s in at[1]], torch.int64), pages.cache, pages.table.cuda(),
                  device_int(pages.lens), device_int(starts), max(new), max(pages.lens))
        for b in range(len(new)):
            outs[b].append(y[starts[b]:starts[b + 1]])
    return [torch.cat(o) for o in outs]


class Decoder:
    """One token of every sequence a call, replayed from a CUDA graph: the
    host writes the step's inputs into buffers that the graph reads."""

    def __init__(self, block, pages, hidden):
        seqs = len(pages.lens)
        self.block, self.pages = block, pages
        self.x = torch.zeros((seqs, hidden), dtype=torch.bfloat16, device="cuda")
        self.positions, self.lens = device_int([0] * seqs), device_int([0] * seqs)
        self.slots = device_int([-1] * seqs, torch.int64)  # padded tokens: the warm-up appends nothing
        self.table = pages.table.cuda()
        self.step()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = self.step()

    def step(self):
        return self.block(self.x, self.positions, self.slots, self.pages.cache, self.table, self.lens)

    def __call__(self, x):
        placed = [self.pages.grow(b, 1) for b in range(len(x))]
        self.x.copy_(x)
        self.positions.copy_(torch.tensor([at[0][0] for at in placed], dtype=torch.int32))
        self.slots.copy_(torch.tensor([at[1][0] for at in placed], dtype=torch.int64))
        self.lens.copy_(torch.tensor(self.pages.lens, dtype=torch.int32))
        self.table.copy_(self.pages.table)
        self.graph.replay()
        return self.y.clone()


def build(heads=32, kv_heads=8, head_dim=128, hidden=4096, page=16, prompts=(700, 33, 1024), steps=8, codes=False, seed=7):
    """A block of random weights, its pages, and random inputs."""
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    rows = (heads + 2 * kv_heads) * head_dim
    wqkv = torch.randn((rows, hidden), generator=g, device="cuda") * hidden ** -0.5
    wo = torch.randn((hidden, heads * head_dim), generator=g, device="cuda") * (heads * head_dim) ** -0.5
    longest = max(prompts) + steps
    block = AttentionBlock(wqkv, wo, heads, kv_heads, head_dim, fw.Rope(rope_table(longest, head_dim)))
    pages = Pages(sum(-(-(p + steps) // page) for p in prompts) + 4, page, kv_heads, head_dim, len(prompts), -(-longest // page), codes)
    x = [torch.randn((p + steps, hidden), generator=g, device="cuda").bfloat16() for p in prompts]
    return block, pages, x


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--codes", action="store_true", help="e4m3 cache")
    ap.add_argument("--steps", type=int, default=64)
    args = ap.parse_args()
    block, pages, x = build(steps=args.steps, codes=args.codes)
    prompts = [t[:len(t) - args.steps] for t in x]
    prefill(block, pages, prompts, 512)
    decode = Decoder(block, pages, x[0].shape[1])
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    used = 0.0
    for i in range(args.steps):
        step = torch.stack([t[len(p) + i] for t, p in zip(x, prompts)])
        start.record()
        decode(step)
        end.record()
        end.synchronize()
        used += start.elapsed_time(end)
    if fw.device_error():
        raise RuntimeError("a kernel gave up: %d" % fw.device_error())
    print("%d sequences of %s tokens, %s cache: %.1f us a decoding step of the block, with its inputs' copies" %
          (len(x), pages.lens, "e4m3" if args.codes else "bf16", used / args.steps * 1e3))


if __name__ == "__main__":
    main()
