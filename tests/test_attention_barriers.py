"""The softmax warps of csrc/attention.cu meet in named barriers, which have no
time limit, while each of their waits on an mbarrier has one.  So no barrier may
stand behind what a wait came to: this reads the source and follows its blocks.
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
    """(heads of the blocks around it, statement) of each statement; an `if`
    without a block is part of its statement, the condition first."""
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
            if c == "{":
                heads.append(part)
            else:
                if part:
                    yield list(heads), part
                if c == "}":
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


def test_no_softmax_barrier_depends_on_a_wait():
    text = source()
    softmax = section(text, "reg_up<L::kRegsSoftmax>()", "tc_fence_before();\n    if (p.cl > 1)")
    join = section(text, "__noinline__ void join_results", "\n}\n") + "\n}"
    # the section starts inside the role's block and ends with the kernel's
    softmax = "void softmax() {" + softmax.rstrip().rstrip("}") + "}"
    for part in (softmax, join):
        assert BARRIER.search(part)
        assert faults(part) == []


def test_all_threads_agree_on_whether_there_is_work():
    have = re.search(r"const bool have = ([^;]*);", source())[1]
    assert "abort_flag" not in have
