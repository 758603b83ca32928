"""The calls of the 4-bit form refuse bad arguments on the host, before any CUDA
call (fake device addresses: no GPU needed)."""
import ctypes

import pytest

import fp8_weight_only_gb300 as fw
from tests import test_abi_cache as cache_tests

P = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(8)]


def at(x):
    return ctypes.c_void_p(x)


def quantize(w=P[0], kind=3, n=4, k=64, codes=P[1], blocks=P[2], scales=P[3]):
    return fw.lib().fp8w_quantize_fp4(w, kind, n, k, codes, blocks, scales, None)


def dequantize(codes=P[1], blocks=P[2], scales=P[3], n=4, k=64, kind=1, w=P[0]):
    return fw.lib().fp8w_dequantize_fp4(codes, blocks, scales, n, k, kind, w, None)


def linear(x=P[0], act=1, m=2, k=64, codes=P[1], blocks=P[2], scales=P[3], bias=None, n=8, y=P[4], flags=0):
    return fw.lib().fp8w_linear_fp4(x, act, m, k, codes, blocks, scales, bias, n, y, flags, None)


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), 1), (dict(codes=None), 1), (dict(blocks=None), 1), (dict(scales=None), 1),
    (dict(kind=0), 4), (dict(kind=4), 4), (dict(kind=5), 4),
    (dict(n=0), 2), (dict(n=2 ** 31), 2), (dict(k=0), 2), (dict(k=16), 2), (dict(k=48), 2), (dict(k=65536 + 32), 2), (dict(k=-32), 2),
    (dict(w=at(0x100008)), 3), (dict(codes=at(0x200004)), 3), (dict(blocks=at(0x300008)), 3), (dict(scales=at(0x400002)), 3),
])
def test_quantize_rejects_bad_arguments(kw, status):
    assert quantize(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), 1), (dict(codes=None), 1), (dict(blocks=None), 1), (dict(scales=None), 1),
    (dict(kind=0), 4), (dict(kind=5), 4), (dict(n=0), 2), (dict(k=48), 2), (dict(k=65536 + 32), 2),
    (dict(w=at(0x100008)), 3), (dict(codes=at(0x200008)), 3), (dict(blocks=at(0x300001)), 3), (dict(scales=at(0x400001)), 3),
])
def test_dequantize_rejects_bad_arguments(kw, status):
    assert dequantize(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(codes=None), 1), (dict(blocks=None), 1), (dict(scales=None), 1), (dict(y=None), 1),
    (dict(act=0), 4), (dict(act=3), 4), (dict(act=5), 4),
    (dict(m=0), 2), (dict(n=0), 2), (dict(k=16), 2), (dict(k=80), 2), (dict(k=65536 + 32), 2), (dict(m=2 ** 31), 2),
    (dict(x=at(0x100002)), 3), (dict(codes=at(0x200008)), 3), (dict(blocks=at(0x300004)), 3), (dict(scales=at(0x400002)), 3),
    (dict(bias=at(0x600001)), 3), (dict(y=at(0x500001)), 3), (dict(flags=2), 6), (dict(flags=-1), 6),
])
def test_linear_rejects_bad_arguments(kw, status):
    assert linear(**kw) == status


def cache(**kw):
    a = dict(k=0x500000, v=0x600000, ks=0x700000, vs=0x800000, pages=10, page_stride=2 * 16 * 32, head_stride=16 * 32, token_stride=32,
             dtype=5, kv_heads=2, dim=64, page=16, kb=0x900000, vb=0xA00000)
    a.update(kw)
    return fw.KVCacheSpec(a["k"], a["v"], a["ks"], a["vs"], a["pages"], a["page_stride"], a["head_stride"], a["token_stride"],
                          a["dtype"], a["kv_heads"], a["dim"], a["page"], a["kb"], a["vb"])


CACHES = [
    (dict(k=None), 1), (dict(ks=None), 1), (dict(vs=None), 1), (dict(kb=None), 1), (dict(vb=None), 1),
    (dict(dtype=4), 7),                                  # blocks with e4m3 codes
    (dict(dtype=1, ks=None, vs=None), 7),                # and with 16-bit values
    (dict(dtype=6), 4), (dict(dim=48), 2), (dict(dim=80), 2), (dict(dim=16), 2), (dict(dim=160), 2), (dict(page=8), 2),
    (dict(token_stride=16), 7), (dict(head_stride=16), 7), (dict(page_stride=31), 7),
    (dict(token_stride=40), 3), (dict(head_stride=520), 3), (dict(page_stride=1032), 3), (dict(k=0x500008), 3), (dict(v=0x600004), 3),
    (dict(ks=0x700002), 3), (dict(kb=0x900002), 3), (dict(vb=0xA00008), 3),
]


@pytest.mark.parametrize("kw,status", CACHES)
def test_append_and_attention_reject_a_bad_cache(kw, status):
    assert cache_tests.append(cache=cache(**kw)) == status
    assert cache_tests.attention(cache=cache(**kw)) == status


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    w, b = torch.zeros((4, 64)), torch.zeros((4, 32), dtype=torch.uint8)
    with pytest.raises(TypeError):
        fw.quantize_fp4(w)
    with pytest.raises(TypeError):
        fw.dequantize_fp4(b, torch.zeros((4, 4), dtype=torch.uint8), torch.zeros(4))
    with pytest.raises(TypeError):
        fw.linear_fp4(w.bfloat16(), b, torch.zeros((4, 4), dtype=torch.uint8), torch.zeros(4))
