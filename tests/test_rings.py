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
template <int NT, bool kFp4> static void skinny(int* out) {
    using R = SkinnyRings<NT, kFp4>;
    out[0] = R::kLanes, out[1] = R::kMmaWarps, out[2] = R::kASlotsAll, out[3] = R::kReady, out[4] = R::kCodeSlots, out[5] = R::kXSlots;
    out[6] = R::kDBuf, out[7] = R::kDoneSlots;
}
extern "C" void skinny_rings(int nt, int fp4, int* out) {
    if (fp4)
        nt == 16 ? skinny<16, true>(out) : nt == 32 ? skinny<32, true>(out) : skinny<64, true>(out);
    else
        nt == 16 ? skinny<16, false>(out) : nt == 32 ? skinny<32, false>(out) : skinny<64, false>(out);
}
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
    """K4: one CTA with `tiles` tiles of nkb k-blocks of 64, as many of them a code stage
    as there are dequantising warpgroups (4 bits: four)."""
    ncs = -(-nkb // groups)
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
                j = groups * cs + h
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


def prefill_faults(rings, bn, nkb, part, runs, tiles=4, groups=None):
    pcs, pas, pxs, four = numbers(rings.prefill_rings, bn)[:4]
    groups = groups or four
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


@pytest.mark.parametrize("bn", [128, 256])
def test_prefill_of_eight_bits(rings, bn):
    # two warpgroups, the same part of a stage in every tile: at most three k-blocks on, one less than the ring
    for nkb in range(1, 21):
        assert prefill_faults(rings, bn, nkb, lambda group, before: group, 20, groups=2) == [], nkb


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


def skinny_roles(tiles, lanes, mma_warps, slots, ready, code_slots, x_slots, dbuf, done_slots, seed):
    """K3 with scales a row (or 4 bits): one CTA, tiles of so many units each."""
    units = sum(tiles)
    ends = [sum(tiles[:i + 1]) - 1 for i in range(len(tiles))]
    cfull = [[Bar("cfull%d,%d" % (g, s), 1) for s in range(code_slots)] for g in range(lanes)]
    cempty = [[Bar("cempty%d,%d" % (g, s), WARPS) for s in range(code_slots)] for g in range(lanes)]
    aready, done = [Bar("aready%d" % i, WARPS) for i in range(ready)], [Bar("done%d" % i, 1) for i in range(done_slots)]
    xfull = [Bar("xfull%d" % s, 1) for s in range(x_slots)]
    dfree = [Bar("dfree%d" % d, 1) for d in range(dbuf)]
    dready = [[Bar("dready%d,%d" % (w, d), 1) for d in range(dbuf)] for w in range(mma_warps)]
    codes = [Slots("codes%d" % g, code_slots, 1) for g in range(lanes)]
    a, x = Slots("A", slots, WARPS), Slots("x", x_slots, 1)
    readers = {}
    c_land, x_land, tensor, sums = Queue(), Queue(), [Queue() for _ in range(mma_warps)], {}

    def code_producer():
        for it in range(units):
            g, j = it % lanes, it // lanes
            s, use = j % code_slots, j // code_slots
            yield wait(cempty[g][s], use & 1 ^ 1, use)

            def land(g=g, s=s, it=it):
                codes[g].put(s, 0, it)
                cfull[g][s].arrive()
            c_land.append(land)
        c_land.ended = True

    def x_producer():
        for it in range(units):
            if it >= x_slots:
                v = it - x_slots
                yield wait(done[v % done_slots], v // done_slots & 1, v // done_slots + 1)

            def land(it=it):
                x.put(it % x_slots, 0, it)
                xfull[it % x_slots].arrive()
            x_land.append(land)
            yield None
        x_land.ended = True

    def dequantiser(group, warp):
        for it in range(group, units, lanes):
            j = it // lanes
            s, use = j % code_slots, j // code_slots
            yield wait(cfull[group][s], use & 1, use + 1)
            if codes[group].held[s][0] != it:
                raise Fault("codes%d slot %d: %s for %d" % (group, s, codes[group].held[s][0], it))
            if it >= slots:
                v = it - slots
                yield wait(done[v % done_slots], v // done_slots & 1, v // done_slots + 1)
            a.put(it % slots, warp, it)
            yield None
            aready[it % ready].arrive()
            readers[it] = readers.get(it, 0) + 1
            if readers[it] == WARPS:
                codes[group].use(s, it)
            cempty[group][s].arrive()

    def mma(w):
        def parts(it):
            return [wait(aready[it % ready], it // ready & 1, it // ready + 1), wait(xfull[it % x_slots], it // x_slots & 1, it // x_slots + 1)]

        if w < units:
            for p in parts(w):
                yield p
        seg, first, issued = 0, True, False
        for it in range(units):
            d = seg % dbuf
            if first:
                yield wait(dfree[d], seg // dbuf & 1 ^ 1, seg // dbuf)
            first = False
            if it % mma_warps == w:
                # the next unit's barriers are asked before this unit's products
                missing = []
                if it + mma_warps < units:
                    for p in parts(it + mma_warps):
                        if not p[0].passes(p[1]):
                            missing.append(p)
                        elif p[0].over < p[2]:
                            raise Fault("%s: passes with %d phases over, for %d" % (p[0].name, p[0].over, p[2]))
                tensor[w].append((seg, it))
                issued = True
                yield None
                for p in missing:
                    yield p
            if it == ends[seg]:
                if issued:
                    tensor[w].append((seg, None))
                else:
                    dready[w][d].arrive()
                yield None
                seg, first, issued = seg + 1, True, False
        tensor[w].ended = True

    def tensor_core(w):
        while True:
            yield tensor[w], 0, 0
            if not tensor[w].items:
                return
            seg, it = tensor[w].items.pop(0)
            if it is None:
                dready[w][seg % dbuf].arrive()
            else:
                a.use(it % slots, it)
                x.use(it % x_slots, it)
                sums.setdefault(seg, []).append(it)
                done[it % done_slots].arrive()

    def epilogue():
        for seg in range(len(tiles)):
            for w in range(mma_warps):
                yield wait(dready[w][seg % dbuf], seg // dbuf & 1, seg // dbuf + 1)
            if sorted(sums.get(seg, [])) != list(range(ends[seg] + 1 - tiles[seg], ends[seg] + 1)):
                raise Fault("tile %d: %s" % (seg, sums.get(seg)))
            yield None
            dfree[seg % dbuf].arrive()

    roles = [code_producer(), x_producer(), copier(c_land, seed), copier(x_land, ~seed), epilogue()]
    roles += [f(w) for w in range(mma_warps) for f in (mma, tensor_core)]
    return roles + [dequantiser(g, w) for g in range(lanes) for w in range(WARPS)]


UNITS = ([1], [2], [3], [5], [16], [1, 1, 1, 1, 1], [2, 2, 2], [3, 1, 4, 1, 5], [4, 4, 4], [7, 7, 7, 7], [13, 20, 6])


def skinny_faults(numbers_, tiles, runs):
    found = []
    for seed in range(runs):
        try:
            play(skinny_roles(tiles, *numbers_, seed), seed)
        except Fault as f:
            found.append(str(f))
    return found


@pytest.mark.parametrize("nt", [16, 32, 64])
@pytest.mark.parametrize("fp4", [1, 0])
def test_skinny(rings, nt, fp4):
    n = numbers(rings.skinny_rings, nt, fp4)
    for tiles in UNITS:
        assert skinny_faults(n, tiles, 20) == [], tiles


@pytest.mark.parametrize("nt", [16, 32, 64])
def test_the_model_sees_barriers_that_change_their_mma_warp(rings, nt):
    # a barrier for each of three slots, which two warps wait for in turn
    n = numbers(rings.skinny_rings, nt, 1)
    n[3] = n[2]
    assert n[3] == 3
    for tiles in ([5], [16], [4, 4, 4], [3, 1, 4, 1, 5]):
        assert skinny_faults(n, tiles, 20), tiles
