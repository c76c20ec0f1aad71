"""The kernels' bounded waits, read from their sources. A wait that gives up makes its thread leave a loop. Where one thread
waits (a loader), that is its own affair. Where a whole warp waits, each thread would judge for itself whether the barrier
came in time; were they to differ, some would leave and the others stop in the next instruction that takes all 32, for
good. So a warp's waits are mbar_wait_bounded_warp, which agrees on the outcome."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_precision_bsq_gb300", "csrc")
SOURCES = sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh")))
ONE_THREAD = re.compile(r"\blane == 0\b|\bthreadIdx\.x == 0\b")


def code_of(text):
    return re.sub(r"//[^\n]*|/\*.*?\*/", lambda m: re.sub(r"[^\n]", " ", m.group()), text, flags=re.S)


def blocks_around(code, at):
    """What stands ahead of each brace that is open at `at`, outermost first."""
    heads, start = [], 0
    for i, c in enumerate(code[:at]):
        if c == "{":
            heads.append(code[start:i])
            start = i + 1
        elif c == "}":
            heads.pop()
            start = i + 1
        elif c == ";":
            start = i + 1 if code[start:i].count("(") == code[start:i].count(")") else start
    return heads


def waits_that_leave(code):
    """Places of a thread's own bounded waits whose outcome decides on a way."""
    for m in re.finditer(r"\bmbar_wait_bounded\s*\(", code):
        line = code[code.rfind("\n", 0, m.start()) + 1:m.start()]
        ahead = re.split(r"[;{}]", code[:m.start()])[-1]
        if "__device__" in ahead or "__all_sync" in ahead:  # its definition, and the warp's form of it
            continue
        if ahead.strip():  # `if (!wait)`, `ok = wait`: not a statement of its own
            yield m.start(), line


@pytest.mark.parametrize("name", SOURCES)
def test_only_single_threads_wait_for_themselves(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        code = code_of(f.read())
    for at, line in waits_that_leave(code):
        assert any(ONE_THREAD.search(h) for h in blocks_around(code, at)), \
            "%s:%d: a warp's wait without a vote: %s" % (name, code.count("\n", 0, at) + 1, line.strip())


def test_the_rule_tells_them_apart():
    alone = "void f() { if (warp == 0 && lane == 0) { for (;;) { if (!mbar_wait_bounded(b, 0)) break; } } }"
    warp = "void f() { if (warp == 1) { for (;;) { if (!mbar_wait_bounded(b, 0)) break; } } }"
    behind = "void f() { if (lane == 0) { g(); } if (!mbar_wait_bounded(b, 0)) return; }"
    agreed = "void f() { if (!mbar_wait_bounded_warp(b, 0)) return; mbar_wait_bounded(drain, 0); }"
    for code, found, single in ((alone, 1, True), (warp, 1, False), (behind, 1, False), (agreed, 0, True)):
        waits = list(waits_that_leave(code))
        assert len(waits) == found
        assert all(any(ONE_THREAD.search(h) for h in blocks_around(code, at)) for at, _ in waits) == single
    assert any("mbar_wait_bounded_warp" in open(os.path.join(CSRC, n), encoding="utf-8").read() for n in SOURCES)
