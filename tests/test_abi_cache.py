"""fp8w_rope, fp8w_rope_append and fp8w_paged_attention refuse bad arguments on
the host, before any CUDA call (fake device addresses: no GPU needed)."""
import ctypes

import pytest

import fp8_weight_only_gb300 as fw

P = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(10)]


def at(x):
    return ctypes.c_void_p(x)


def rope_spec(**kw):
    a = dict(table=0x900000, max_pos=100, rot_dim=64, interleaved=0, axes=1, sections=(32, 0, 0, 0))
    a.update(kw)
    return fw.RopeSpec(a["table"], a["max_pos"], a["rot_dim"], a["interleaved"], a["axes"], (ctypes.c_int * 4)(*a["sections"]))


SPECS = [
    (dict(table=0), 1), (dict(rot_dim=0, sections=(0, 0, 0, 0)), 2), (dict(rot_dim=24, sections=(12, 0, 0, 0)), 2),
    (dict(rot_dim=80, sections=(40, 0, 0, 0)), 2), (dict(max_pos=0), 7), (dict(axes=0), 7), (dict(axes=5), 7),
    (dict(sections=(31, 0, 0, 0)), 7), (dict(sections=(16, 16, 0, 0)), 7), (dict(axes=2, sections=(40, -8, 0, 0)), 7),
    (dict(table=0x900008), 3),
]


def rope(x=P[0], act=1, tokens=4, heads=2, dim=64, xs=128, pos=P[1], spec=None, y=P[2], ys=128, null_spec=False):
    s = rope_spec() if spec is None else spec
    return fw.lib().fp8w_rope(x, act, tokens, heads, dim, xs, pos, None if null_spec else ctypes.byref(s), y, ys, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(y=None), 1), (dict(pos=None), 1), (dict(null_spec=True), 1),
    (dict(act=0), 4), (dict(act=3), 4), (dict(act=4), 4),
    (dict(tokens=0), 2), (dict(tokens=-1), 2), (dict(tokens=2 ** 31), 2), (dict(heads=0), 2), (dict(dim=72, xs=144, ys=144), 2),
    (dict(dim=8), 2), (dict(dim=272, xs=544, ys=544), 2),
    (dict(xs=127), 7), (dict(ys=64), 7), (dict(xs=132), 3), (dict(ys=129), 3), (dict(x=at(0x100008)), 3),
    (dict(y=at(0x300002)), 3), (dict(pos=at(0x200002)), 3), (dict(y=P[0], ys=256), 7),
])
def test_rope_rejects_bad_arguments(kw, status):
    assert rope(**kw) == status


@pytest.mark.parametrize("kw,status", SPECS)
def test_rope_rejects_a_bad_spec(kw, status):
    assert rope(spec=rope_spec(**kw)) == status


def cache_spec(**kw):
    a = dict(k=0x500000, v=0x600000, ks=None, vs=None, pages=10, page_stride=2 * 16 * 64, head_stride=16 * 64, token_stride=64,
             dtype=1, kv_heads=2, dim=64, page=16)
    a.update(kw)
    return fw.KVCacheSpec(a["k"], a["v"], a["ks"], a["vs"], a["pages"], a["page_stride"], a["head_stride"], a["token_stride"],
                          a["dtype"], a["kv_heads"], a["dim"], a["page"])


CACHES = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(dtype=4), 1), (dict(dtype=4, ks=0x700000), 1),
    (dict(dtype=2), 4), (dict(dtype=3), 4), (dict(dtype=0), 4),
    (dict(pages=0), 2), (dict(pages=2 ** 31), 2), (dict(kv_heads=0), 2), (dict(dim=72), 2), (dict(dim=144), 2), (dict(dim=0), 2),
    (dict(page=0), 2), (dict(page=8), 2), (dict(page=24), 2), (dict(page=512), 2),
    (dict(token_stride=48), 7), (dict(head_stride=0), 7), (dict(page_stride=-2048), 7), (dict(page_stride=2 ** 40), 7),
    (dict(ks=0x700000), 7),
    (dict(token_stride=68), 3), (dict(head_stride=1028), 3), (dict(page_stride=2049), 3), (dict(k=0x500008), 3), (dict(v=0x600004), 3),
    (dict(dtype=4, ks=0x700002, vs=0x800000), 3), (dict(dtype=4, ks=0x700000, vs=0x800001), 3),
    (dict(dtype=4, ks=0x700000, vs=0x800000, token_stride=72), 3),
]


def append(q=P[0], k=P[1], v=P[2], act=1, tokens=4, heads=4, qs=256, ks=128, vs=128, pos=P[3], spec=None, slots=P[4], cache=None,
           out=P[5], os_=256, no_spec=False, no_cache=False):
    s, c = rope_spec() if spec is None else spec, cache_spec() if cache is None else cache
    return fw.lib().fp8w_rope_append(q, k, v, act, tokens, heads, qs, ks, vs, pos, None if no_spec else ctypes.byref(s), slots,
                                     None if no_cache else ctypes.byref(c), out, os_, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(no_cache=True), 1), (dict(out=None), 1), (dict(pos=None), 1),
    (dict(act=3), 4), (dict(act=2), 4), (dict(tokens=0), 2), (dict(heads=0), 2),
    (dict(qs=255), 7), (dict(ks=64), 7), (dict(vs=127), 7), (dict(os_=8), 7), (dict(out=P[0], os_=512), 7),
    (dict(qs=260), 3), (dict(ks=130), 3), (dict(vs=132), 3), (dict(os_=257), 3), (dict(k=at(0x200008)), 3),
    (dict(slots=at(0x500004)), 3), (dict(q=at(0x100002)), 3),
    (dict(q=None, ks=64), 7), (dict(no_spec=True, vs=1), 7),
])
def test_rope_append_rejects_bad_arguments(kw, status):
    assert append(**kw) == status


@pytest.mark.parametrize("kw,status", CACHES)
def test_rope_append_rejects_a_bad_cache(kw, status):
    assert append(cache=cache_spec(**kw)) == status


@pytest.mark.parametrize("kw,status", SPECS)
def test_rope_append_rejects_a_bad_spec(kw, status):
    assert append(spec=rope_spec(**kw)) == status


def attention(q=P[0], act=1, tokens=4, heads=4, qs=256, cache=None, table=P[1], width=8, lens=P[2], starts=P[3], seqs=2, scale=0.1,
              window=0, max_new=0, max_len=0, out=P[4], os_=256, no_cache=False):
    c = cache_spec() if cache is None else cache
    return fw.lib().fp8w_paged_attention(q, act, tokens, heads, qs, None if no_cache else ctypes.byref(c), table, width, lens, starts,
                                         seqs, scale, window, max_new, max_len, out, os_, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(out=None), 1), (dict(no_cache=True), 1),
    (dict(act=3), 4), (dict(act=2), 4),
    (dict(tokens=0), 2), (dict(seqs=0), 2), (dict(heads=0), 2), (dict(heads=3), 2), (dict(width=0), 2), (dict(width=2 ** 27), 2),
    (dict(starts=None), 2), (dict(tokens=2 ** 30), 2),
    (dict(scale=0.0), 7), (dict(scale=-1.0), 7), (dict(scale=float("inf")), 7), (dict(scale=float("nan")), 7),
    (dict(window=-1), 7), (dict(max_new=-1), 7), (dict(max_len=-5), 7), (dict(qs=255), 7), (dict(os_=200), 7),
    (dict(qs=258), 3), (dict(os_=260), 3), (dict(q=at(0x100008)), 3), (dict(out=at(0x500002)), 3),
    (dict(table=at(0x200002)), 3), (dict(lens=at(0x300001)), 3), (dict(starts=at(0x400002)), 3),
])
def test_paged_attention_rejects_bad_arguments(kw, status):
    assert attention(**kw) == status


@pytest.mark.parametrize("kw,status", CACHES)
def test_paged_attention_rejects_a_bad_cache(kw, status):
    assert attention(cache=cache_spec(**kw)) == status


def test_value_error_has_a_name():
    assert fw.lib().fp8w_status_string(7) != b"unknown status"


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    page = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fw.Rope(torch.zeros((4, 64)))
    with pytest.raises(TypeError):
        fw.KVCache(page, page)
    with pytest.raises(TypeError):
        fw.rope(x, torch.zeros(2, dtype=torch.int32), None)
