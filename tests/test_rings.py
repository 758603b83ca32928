"""A model of the barriers of the tensor-core kernels, on the numbers and functions of
csrc/rings.h (built with the host compiler): every role is a process that waits for
phases by their parity, as on the device, and the processes take their steps in random
orders, some of them far behind the others.  A run fails where a wait passes before
the phase that it is for is over, where an operand is overwritten or multiplied too
early, and where all processes wait.  (A race shows on a GPU only now and then; in the
model an order that lets it happen is one of those drawn.)"""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_weight_only_gb300", "csrc")
WARPS = 2          # of a warpgroup (4 on the device)


@pytest.fixture(scope="module")
def rings(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    at = tmp_path_factory.mktemp("rings")
    src = at / "rings.cpp"
    src.write_text(SOURCE)
    lib = at / "rings.so"
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(str(lib))


SOURCE = r"""
#include "rings.h"
using namespace fp8w;
template <int BN> static void prefill(int* out) {
    out[0] = PrefillRings<BN>::kPCS, out[1] = PrefillRings<BN>::kPAS, out[2] = PrefillRings<BN>::kPXS, out[3] = kPFp4Groups;
}
extern "C" void prefill_rings(int bn, int* out) { bn == 128 ? prefill<128>(out) : prefill<256>(out); }
extern "C" int part(int group, long long before) { return prefill_fp4_part(group, before); }
"""


def numbers(call, *args, count=8):
    out = (ctypes.c_int * count)()
    call(*args, out)
    return list(out)


class Fault(Exception):
    pass


class Bar:
    def __init__(self, name, arrivals):
        self.name, self.arrivals, self.left, self.over = name, arrivals, arrivals, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.over = self.arrivals, self.over + 1

    def passes(self, parity):     # the phase that is on is not of this parity
        return (self.over & 1) != parity


def wait(bar, parity, needs):
    """A wait by parity that means: `needs` phases are over."""
    return bar, parity, needs


def play(roles, seed):
    """The roles (generators of waits, None for a step of other work) in an order of
    the seed's: a role's chance of the next step is drawn anew now and then, over four
    powers of ten."""
    rng = random.Random(seed)
    live = [(r, next(r, False)) for r in roles]
    live = [x for x in live if x[1] is not False]
    chance, turn = {}, 0
    while live:
        if turn % 60 == 0:
            chance = {id(r): 10.0 ** rng.uniform(-4, 0) for r, _ in live}
        turn += 1
        ready = [i for i, (_, w) in enumerate(live) if w is None or w[0].passes(w[1])]
        if not ready:
            raise Fault("all wait: " + ", ".join(w[0].name for _, w in live))
        i = rng.choices(ready, [chance[id(live[i][0])] for i in ready])[0]
        role, w = live[i]
        if w is not None and w[0].over < w[2]:
            raise Fault("%s: passes with %d phases over, for %d" % (w[0].name, w[0].over, w[2]))
        w = next(role, False)
        if w is False:
            live.pop(i)
        else:
            live[i] = role, w


class Slots:
    """What a ring's slots hold, by the parts of a slot that different warps write."""

    def __init__(self, name, slots, parts):
        self.name, self.held, self.used = name, [[None] * parts for _ in range(slots)], [True] * slots

    def put(self, slot, part, what):
        if not self.used[slot] and self.held[slot][part] is not None:
            raise Fault("%s slot %d: %s over %s" % (self.name, slot, what, self.held[slot][part]))
        if self.used[slot]:
            self.held[slot], self.used[slot] = [None] * len(self.held[slot]), False
        self.held[slot][part] = what

    def use(self, slot, what):
        if any(h != what for h in self.held[slot]):
            raise Fault("%s slot %d: %s for %s" % (self.name, slot, self.held[slot], what))
        self.used[slot] = True


class Queue:
    """Work handed to an engine, which waits while there is none."""
    name, over = "queue", float("inf")

    def __init__(self):
        self.items, self.ended = [], False

    def append(self, item):
        self.items.append(item)

    def passes(self, parity):
        return bool(self.items) or self.ended


def copier(landing, seed):
    """Copies in flight, which land in an order of the run's."""
    rng = random.Random(seed)
    while True:
        yield landing, 0, 0
        if not landing.items:
            return
        landing.items.pop(rng.randrange(len(landing.items)))()


def prefill_roles(nkb, tiles, pcs, pas, pxs, groups, part, seed):
    """K4's 4-bit form: one CTA with `tiles` tiles of nkb k-blocks of 64."""
    ncs = -(-nkb // 4)
    cfull, cempty = [Bar("cfull%d" % s, 1) for s in range(pcs)], [Bar("cempty%d" % s, groups * WARPS) for s in range(pcs)]
    afull, aempty = [Bar("afull%d" % s, WARPS) for s in range(pas)], [Bar("aempty%d" % s, 1) for s in range(pas)]
    xfull, xempty = [Bar("xfull%d" % s, 1) for s in range(pxs)], [Bar("xempty%d" % s, 1) for s in range(pxs)]
    dfull, dempty = [Bar("dfull%d" % d, 1) for d in range(2)], [Bar("dempty%d" % d, 1) for d in range(2)]
    codes, a, x = Slots("codes", pcs, 1), Slots("A", pas, WARPS), Slots("x", pxs, 1)
    readers = [0] * pcs           # warps that have read a code slot
    c_land, x_land, tensor, sums = Queue(), Queue(), Queue(), {}

    def code_producer():
        for i in range(tiles * ncs):
            s = i % pcs
            yield wait(cempty[s], (i // pcs & 1) ^ 1, i // pcs)

            def land(s=s, i=i):
                codes.put(s, 0, i)
                cfull[s].arrive()
            c_land.append(land)
        c_land.ended = True

    def x_producer():
        for i in range(tiles * nkb):
            s = i % pxs
            yield wait(xempty[s], (i // pxs & 1) ^ 1, i // pxs)

            def land(s=s, i=i):
                x.put(s, 0, i)
                xfull[s].arrive()
            x_land.append(land)
        x_land.ended = True

    def dequantiser(group, warp):
        base = 0
        for t in range(tiles):
            h = part(group, base)
            for cs in range(ncs):
                i = t * ncs + cs
                s = i % pcs
                yield wait(cfull[s], i // pcs & 1, i // pcs + 1)
                if codes.held[s][0] != i:
                    raise Fault("codes slot %d: %s for %d" % (s, codes.held[s][0], i))
                j = 4 * cs + h
                if j < nkb:
                    kb = base + j
                    yield wait(aempty[kb % pas], (kb // pas & 1) ^ 1, kb // pas)
                    a.put(kb % pas, warp, kb)
                    yield None
                    afull[kb % pas].arrive()
                readers[s] += 1
                if readers[s] == groups * WARPS:
                    readers[s] = 0
                    codes.use(s, i)
                cempty[s].arrive()
            base += nkb

    def mma():
        kb = 0
        for t in range(tiles):
            d = t & 1
            yield wait(dempty[d], (t >> 1 & 1) ^ 1, t >> 1)
            for j in range(nkb):
                sa, sx = kb % pas, kb % pxs
                yield wait(afull[sa], kb // pas & 1, kb // pas + 1)
                yield wait(xfull[sx], kb // pxs & 1, kb // pxs + 1)
                tensor.append((t, kb, sa, sx))
                kb += 1
            tensor.append((t, None, None, None))
        tensor.ended = True

    def tensor_core():
        while True:
            yield tensor, 0, 0
            if not tensor.items:
                return
            t, kb, sa, sx = tensor.items.pop(0)
            if kb is None:
                dfull[t & 1].arrive()
            else:
                a.use(sa, kb)
                x.use(sx, kb)
                sums.setdefault(t, []).append(kb)
                aempty[sa].arrive()
                xempty[sx].arrive()

    def epilogue():
        for t in range(tiles):
            yield wait(dfull[t & 1], t >> 1 & 1, (t >> 1) + 1)
            if sums.get(t) != list(range(t * nkb, (t + 1) * nkb)):
                raise Fault("tile %d: %s" % (t, sums.get(t)))
            yield None
            dempty[t & 1].arrive()

    roles = [code_producer(), x_producer(), copier(c_land, seed), copier(x_land, ~seed), mma(), tensor_core(), epilogue()]
    return roles + [dequantiser(g, w) for g in range(groups) for w in range(WARPS)]


def prefill_faults(rings, bn, nkb, part, runs, tiles=4):
    pcs, pas, pxs, groups = numbers(rings.prefill_rings, bn)[:4]
    found = []
    for seed in range(runs):
        try:
            play(prefill_roles(nkb, tiles, pcs, pas, pxs, groups, part, seed), seed)
        except Fault as f:
            found.append(str(f))
    return found


@pytest.mark.parametrize("bn", [128, 256])
def test_prefill_of_four_bits(rings, bn):
    for nkb in range(1, 21):
        assert prefill_faults(rings, bn, nkb, rings.part, 20) == [], nkb


def test_the_model_sees_a_warpgroup_that_changes_its_stage(rings):
    # the same part of a code stage in every tile: right for multiples of four k-blocks alone
    for nkb in (5, 6, 7, 9, 14, 18):
        assert prefill_faults(rings, 128, nkb, lambda group, before: group, 12), nkb
    for nkb in (4, 8, 16):
        assert not prefill_faults(rings, 128, nkb, lambda group, before: group, 4), nkb


def test_each_k_block_has_one_warpgroup(rings):
    groups = numbers(rings.prefill_rings, 128)[3]
    for nkb in range(1, 21):
        taken = [(t * nkb + 4 * cs + rings.part(g, t * nkb), g) for t in range(5) for cs in range(-(-nkb // 4)) for g in range(groups)
                 if 4 * cs + rings.part(g, t * nkb) < nkb]
        assert sorted(kb for kb, _ in taken) == list(range(5 * nkb))
        assert all(kb % groups == g for kb, g in taken)
