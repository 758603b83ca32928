"""The 4-bit form on the CPU, shared by its tests: the quantiser's rule in fp32
steps (bit for bit what the library has to give), its values in 64 bits, and a
paged cache in it.

    value = scale * e4m3(block) * e2m1(code)
"""
import numpy as np

from tests.attention_reference import Paged

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
F32 = np.float32


def e4m3_values():
    b = np.arange(256)
    e, m, s = (b >> 3) & 15, b & 7, b >> 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v[(b & 127) == 127] = np.nan
    return np.where(s == 1, -v, v)


E4M3 = e4m3_values()


def e4m3_of(x):
    """Nearest-even, saturated e4m3 bytes of non-negative fp32 values."""
    grid = E4M3[:127]
    x = np.minimum(x.astype(np.float64), 448.0)
    hi = np.searchsorted(grid, x)          # first code at or above x
    lo = np.maximum(hi - 1, 0)
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo).astype(np.uint8)


def e2m1_of(y):
    """Nearest-even, saturated e2m1 codes of fp32 values."""
    a = np.minimum(np.abs(y.astype(np.float64)), 6.0)
    hi = np.searchsorted(E2M1, a)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E2M1[lo], E2M1[hi] - a
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return (code + 8 * np.signbit(y)).astype(np.uint8)


def quantize(x):
    """x [..., k] fp32 -> packed codes [..., k / 2], blocks [..., k / 16], scales [...]."""
    x = np.ascontiguousarray(x, dtype=F32)
    amax = np.abs(x).max(-1)
    scales = np.where(amax == 0, F32(1), np.maximum(amax * F32(1 / 2688), F32(2.0 ** -126))).astype(F32)
    y = x * (F32(1) / scales)[..., None]
    parts = y.reshape(*y.shape[:-1], -1, 16)
    blocks = e4m3_of(np.abs(parts).max(-1) * F32(1 / 6))
    b = E4M3[blocks].astype(F32)
    inverse = np.where(b == 0, F32(0), F32(1) / np.where(b == 0, F32(1), b)).astype(F32)
    codes = e2m1_of(parts * inverse[..., None]).reshape(x.shape)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), blocks, scales


def values(codes, blocks, scales):
    """Packed codes, blocks and scales -> the values in 64 bits."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = np.where(c > 7, -E2M1[c & 7], E2M1[c & 7])
    return v * np.repeat(E4M3[blocks], 16, -1) * np.asarray(scales, dtype=np.float64)[..., None]


class Paged4(Paged):
    """A paged cache of 4 bits with random contents; what no sequence owns is NaN
    (scales and blocks) or any code."""

    def __init__(self, torch, fw, seed, lens, kv_heads, dim, page, layout, spare=3, growth=0.0, wide=1, change=None):
        dev = torch.device("cuda:0")
        rng = np.random.default_rng(seed)
        self.lens, self.page = lens, page
        need = [-(-t // page) for t in lens]
        pages = sum(need) + spare
        order = rng.permutation(pages)
        table = np.full((len(lens), max(max(need), 1) + wide), -1, dtype=np.int32)
        codes = rng.integers(0, 256, (2, pages, kv_heads, page, dim // 2), dtype=np.uint8)
        blocks = np.full((2, pages, kv_heads, page, dim // 16), 0x7F, dtype=np.uint8)
        scales = np.full((2, pages, kv_heads, page), np.nan, dtype=F32)
        self.rows, i = [], 0
        for b, t in enumerate(lens):
            own = order[i:i + need[b]]
            i += need[b]
            table[b, :len(own)] = own
            x = rng.standard_normal((2, t, kv_heads, dim)).astype(F32)
            x[0] *= (1.0 + growth * np.arange(t) / max(t, 1))[:, None, None].astype(F32)
            if change is not None:
                change(b, x)
            both = []
            at, off = np.repeat(own, page)[:t], np.arange(t) % page
            for c in range(2):
                got = quantize(x[c]) if t else (np.zeros((0, kv_heads, dim // 2), np.uint8), np.zeros((0, kv_heads, dim // 16), np.uint8), np.zeros((0, kv_heads), F32))
                codes[c][at, :, off], blocks[c][at, :, off], scales[c][at, :, off] = got
                both.append(torch.from_numpy(values(*got)).to(dev))
            self.rows.append(both)
        self.table = torch.from_numpy(table).to(dev)
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device=dev)

        def put(a):
            t = torch.from_numpy(np.ascontiguousarray(a if layout == "heads" else a.swapaxes(1, 2))).to(dev)
            return t if layout == "heads" else t.transpose(1, 2)

        def dense(a):
            return torch.from_numpy(np.ascontiguousarray(a)).to(dev)

        self.cache = fw.KVCache(put(codes[0]), put(codes[1]), dense(scales[0]), dense(scales[1]), dense(blocks[0]), dense(blocks[1]))
