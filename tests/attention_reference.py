"""Attention over a paged cache in 64 bits, and how far the library's outputs
may be from it: shared by the GPU tests of the cache's operators.

The bound of an output element, with A = sum_j p_j |v_j| (the softmax weights
p in 64 bits), u the unit roundoff of the operand type (2^-8 or 2^-11):
  u (A + |o|)                       each weight and the output rounded once
  + 2 e_s A                         scores off by e_s, in numerator and denominator
  + keys 2^-23 A                    fp32 sums, each step truncated at worst
  + keys 2^-24 max|v| / l           (fp16) weights below its normal range, l the sum of exp(s - max)
with e_s = (head_dim + 8) 2^-23 scale max_j sum_d |q_d k_jd| + 2^-18: the
score's sum, its scales and the exponent's argument and approximation.
"""
import numpy as np

ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def attend(torch, q, k, v, n, length, scale, window, dtype):
    """One sequence: q [n, heads, dim], k and v [length, kv_heads, dim] (64
    bits); (out, bound) [n, heads, dim] in 64 bits."""
    heads, kv = q.shape[1], k.shape[1]
    group = heads // kv
    out, tol = torch.zeros_like(q), torch.full_like(q, 0.0)
    if not length:
        return out, tol
    pos = length - n + torch.arange(n, device=q.device)[:, None]
    at = torch.arange(length, device=q.device)[None, :]
    seen = at <= pos
    if window:
        seen &= at > pos - window
    u = ROUND[dtype]
    for h in range(heads):
        kh, vh = k[:, h // group], v[:, h // group]
        s = (q[:, h] @ kh.T) * scale
        s = torch.where(seen, s, torch.full_like(s, -float("inf")))
        top = s.max(-1, keepdim=True).values
        top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        e = torch.where(seen, torch.exp(s - top), torch.zeros_like(s))
        l = e.sum(-1, keepdim=True)
        p = e / torch.where(l == 0, torch.ones_like(l), l)
        o, a = p @ vh, p @ vh.abs()
        e_s = (q.shape[2] + 8) * 2.0 ** -23 * scale * (q[:, h].abs() @ kh.abs().T).max(-1, keepdim=True).values + 2.0 ** -18
        keys = seen.sum(-1, keepdim=True)
        t = u * (a + o.abs()) + 2 * e_s * a + keys * 2.0 ** -23 * a
        if dtype == "f16":
            t = t + keys * 2.0 ** -24 * vh.abs().max() / torch.where(l == 0, torch.ones_like(l), l) + 2.0 ** -25
        out[:, h], tol[:, h] = o, t
    return out, tol


class Paged:
    """A paged cache with random contents: pages in random order, everything
    that no sequence owns (other pages, slots past a length) NaN."""

    def __init__(self, torch, fw, seed, lens, kv_heads, dim, page, dtype, codes, layout, spare=3, growth=0.0, wide=1):
        dev = torch.device("cuda:0")
        g = torch.Generator(dev)
        g.manual_seed(seed)
        self.lens, self.page = lens, page
        need = [-(-t // page) for t in lens]
        pages = sum(need) + spare
        tdt = torch.bfloat16 if dtype == "bf16" else torch.float16
        order = torch.randperm(pages, generator=g, device=dev).tolist()
        table = torch.full((len(lens), max(max(need), 1) + wide), -1, dtype=torch.int32)
        self.rows, i = [], 0
        shape = (pages, kv_heads, page, dim) if layout == "heads" else (pages, page, kv_heads, dim)
        view = (lambda t: t) if layout == "heads" else (lambda t: t.transpose(1, 2))
        nan = 0x7F if codes else float("nan")
        k = view(torch.full(shape, nan, dtype=torch.uint8 if codes else tdt, device=dev))
        v = view(torch.full(shape, nan, dtype=torch.uint8 if codes else tdt, device=dev))
        ks = torch.full((pages, kv_heads, page), float("nan"), device=dev) if codes else None
        vs = ks.clone() if codes else None
        for b, t in enumerate(lens):
            own = order[i:i + need[b]]
            i += need[b]
            table[b, :len(own)] = torch.tensor(own, dtype=torch.int32)
            x = torch.randn((2, t, kv_heads, dim), generator=g, device=dev)
            # keys that grow with their position make the running maximum grow
            x[0] *= (1.0 + growth * torch.arange(t, device=dev) / max(t, 1))[:, None, None]
            both = []
            for c, cache, sc in ((0, k, ks), (1, v, vs)):
                at = torch.tensor(own, device=dev, dtype=torch.int64).repeat_interleave(page)[:t] if t else torch.zeros(0, dtype=torch.int64, device=dev)
                off = torch.arange(t, device=dev) % page
                if codes:
                    s = x[c].abs().amax(-1) / 448.0
                    q = (x[c] / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
                    cache[at, :, off] = q.view(torch.uint8)
                    sc[at, :, off] = s
                    both.append(q.double() * s.double()[..., None])
                else:
                    cache[at, :, off] = x[c].to(tdt)
                    both.append(x[c].to(tdt).double())
            self.rows.append(both)
        self.table = table.to(dev)
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.cache = fw.KVCache(k, v, ks, vs)


def check(torch, got, want, tol):
    """Every element within its bound; returns the largest share of it used."""
    d = (got.double() - want).abs()
    assert bool(torch.isfinite(got).all()), "an output is not finite"
    worst = float((d / tol.clamp_min(1e-300)).max()) if d.numel() else 0.0
    assert bool((d <= tol).all()), "off by up to %.3g of the bound" % worst
    return worst


def bits(t):
    return t.contiguous().view(-1).view({2: __import__("torch").int16, 4: __import__("torch").int32}[t.element_size()]).cpu().numpy().view(
        {2: np.uint16, 4: np.uint32}[t.element_size()])
