"""The softmax warps of csrc/attention.cu meet in named barriers, which have no
time limit, while each of their waits on an mbarrier has one.  So no barrier may
stand behind what a wait came to, and a warp that leaves the loop of tiles when a
wait ran out takes part in the barriers of the tiles left: this reads the source
and follows its blocks.
(A wait that runs out is not made to happen on a GPU: a barrier out of step there
would hang it.)"""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_weight_only_gb300", "csrc", "attention.cu")
BARRIER = re.compile(r"\bBAR_SYNC\b|\b(?:bar_red_or|softmax_bar|exchange|softmax_tile|join_results|cluster_sync_all|__syncthreads)\b\s*(?:<[^;{}]*>)?\s*\(")
OUTCOME = re.compile(r"\bok\b|\ball\b|mbar_wait|abort_flag")
LEAVES = re.compile(r"\b(?:break|return|continue)\b")


def plain(text):
    """Without comments and directives; strings empty, but for those that are a barrier."""
    text = re.sub(r"//[^\n]*|^\s*#[^\n]*", "", text, flags=re.M)
    return re.sub(r'"(?:[^"\\\n]|\\.)*"', lambda m: "BAR_SYNC" if "bar.sync" in m[0] else '""', text)


def section(text, first, last):
    return text[text.index(first):text.index(last, text.index(first))]


def statements(text):
    """(heads of the blocks around it, statement) of each statement and block
    head; an `if` without a block is part of its statement, the condition first."""
    heads, start, depth = [], 0, 0
    for i, c in enumerate(text):
        if c in "([":
            depth += 1
        elif c in ")]":
            depth -= 1
        elif depth:
            continue
        elif c in "{};":
            part = " ".join(text[start:i].split())
            start = i + 1
            if part:
                yield list(heads), part
            if c == "{":
                heads.append(part)
            elif c == "}":
                heads.pop()


def faults(text):
    """Barriers under a condition on a wait's outcome, and statements under one
    that leave a loop (outside of loops, a function) in which there is a barrier."""
    found, blocks = [], list(statements(text))
    for heads, what in blocks:
        if not any(OUTCOME.search(condition(h)) for h in heads + [what]):
            continue
        if BARRIER.search(what):
            found.append(what)
        if LEAVES.search(what):
            loops = [k for k, h in enumerate(heads) if re.match(r"for\b|while\b", h)]
            left = heads[:loops[-1] + 1] if loops else heads[:1]
            if any(h[:len(left)] == left and BARRIER.search(w) for h, w in blocks):
                found.append(what)
    return found


def condition(head):
    """What an `if` or `while` asks, "" for other statements."""
    m = re.search(r"\b(?:if|while)\s*(?:constexpr)?\s*\(", head)
    if not m:
        return ""
    depth, i = 1, m.end()
    while depth:
        depth += {"(": 1, ")": -1}.get(head[i], 0)
        i += 1
    return head[m.end():i - 1]


def source():
    with open(SOURCE) as f:
        return plain(f.read())


def test_the_reader_sees_barriers_behind_a_wait():
    assert faults("void f() { if (ok && busy) { BAR_SYNC; } }")
    assert faults("void f() { for (;;) { if (!mbar_wait_warp(x)) { ok = false; break; } bar_red_or(a, b, c); } }")
    assert faults("void f() { for (;;) { if (!ok) break; softmax_tile(j); } }")
    assert not faults("void f() { for (;;) { if (ok) { ok = mbar_wait_warp(x); } if (busy) softmax_tile(j); if (one) break; } }")


def parts():
    text = source()
    softmax = section(text, "reg_up<L::kRegsSoftmax>()", "tc_fence_before();\n    if (p.cl > 1)")
    # the section starts inside the role's block and ends with the kernel's
    softmax = "void softmax() {" + softmax.rstrip().rstrip("}") + "}"
    return softmax, section(text, "__noinline__ void join_results", "\n}\n") + "\n}"


def test_no_softmax_barrier_depends_on_a_wait():
    softmax, join = parts()
    assert BARRIER.search(softmax) and BARRIER.search(join)
    assert faults(join) == []
    # the loop of tiles, which the next test is about
    assert faults(softmax) == ["break"]


def sequence(text, names):
    """Each barrier of a block, in order: whether it is a vote, and the
    conditions it stands under, by `names` (a condition that is not there fails)."""
    found = []
    for heads, what in statements(text):
        own = condition(what)
        for m in BARRIER.finditer(what):
            around = heads if m[0] in own else heads + [what]
            asked = [names[condition(h)] for h in around if condition(h)]
            found.append(("vote" if m[0].startswith("bar_red_or") else "meet", tuple(asked)))
    return found


def test_a_warp_that_gave_up_takes_the_barriers_of_its_tiles():
    softmax, _ = parts()
    tile = section(softmax, "auto softmax_tile", "const int step =")
    begin = tile.index("auto exchange")
    tile = tile[:begin] + tile[tile.index("float mx"):]      # the calls, without the function itself
    left = section(softmax, "for (; j < jn && busy;", "if (ok && done > 0)")
    names = {"done == 0": "first", "moves": "moved", "W < 64": "copies", "bar_red_or(pair, 64, false)": "moved", "split > 1": "copies"}
    want = [("meet", ("first",)), ("vote", ()), ("meet", ("moved",)), ("meet", ("moved", "copies"))]
    assert sequence(tile, names) == want
    assert sequence(left, names) == want
    # as many tiles, counted alike, by the warps that have rows
    assert "for (; j < jn; j += step, ++done)" in softmax and "for (; j < jn && busy; j += step, ++done)" in softmax
    # copies of the rows are what narrows W
    assert re.search(r"if \(split == 4\)\s*softmax_tile\(std::integral_constant<int, 16>", softmax)
    assert re.search(r"else if \(split == 2\)\s*softmax_tile\(std::integral_constant<int, 32>", softmax)
    assert re.search(r"else\s*softmax_tile\(std::integral_constant<int, 64>", softmax)


def test_all_threads_agree_on_whether_there_is_work():
    have = re.search(r"const bool have = ([^;]*);", source())[1]
    assert "abort_flag" not in have
