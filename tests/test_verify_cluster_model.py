"""The cluster protocol of draft verification
(paged_kv_cache_410_b200/csrc/pa_verify.cuh), model-checked on the CPU.

The cluster operations of the kernel are read from its source in order (the
arrivals, the waits and the stores into the other CTAs' shared memory; those
of the loop once per pass) and make the program of every CTA. CTAs start in
any order and run in any interleaving; a cluster barrier completes when every
CTA has arrived. The checks:

  * no store into a CTA that has not started, or has ended;
  * no pass reads its sums before every CTA has stored them;
  * no state where some CTA waits forever.
"""
import os
import re
from collections import deque

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "paged_kv_cache_410_b200", "csrc", "pa_verify.cuh")


class Violation(Exception):
    pass


def kernel_program(passes, text=None):
    """[op] of one CTA: "arrive", "wait", ("store", pass), ("read", pass)."""
    if text is None:
        with open(SOURCE) as f:
            text = f.read()
    body = text[text.index("pa_verify_kernel(const VerifyParams p)"):]
    body = re.sub(r"//[^\n]*", "", body)
    loop = body.index("for (int attempt")
    ops = re.compile(r"(if \(attempt == 0\) )?(cluster_arrive\(\)|cluster_wait\(\)|st\.shared::cluster)"
                     r"|(double c\[PL\])")
    prog = []

    def add(part, k):
        for m in ops.finditer(part):
            if m.group(3):
                prog.append(("read", k))
            elif m.group(1) and k != 0:
                continue
            elif "arrive" in m.group(2):
                prog.append("arrive")
            elif "wait" in m.group(2):
                prog.append("wait")
            else:
                prog.append(("store", k))

    add(body[:loop], 0)
    for k in range(passes):
        add(body[loop:], k)
    return prog


def check(prog, ctas):
    """Explore every interleaving; returns the number of states."""
    # pc: -1 before the start; arrived: barrier phases a CTA has arrived for
    start = ((-1,) * ctas, (0,) * ctas, (0,) * ctas, frozenset())
    seen, todo = {start}, deque([start])
    while todo:
        pcs, arrived, waited, stored = todo.popleft()
        moved = False
        for c in range(ctas):
            pc = pcs[c]
            if pc == len(prog):
                continue
            a, w, s = list(arrived), list(waited), stored
            if pc >= 0:
                op = prog[pc]
                if op == "arrive":
                    if a[c] != w[c]:
                        raise Violation("a second arrival without a wait")
                    a[c] += 1
                elif op == "wait":
                    if a[c] != w[c] + 1:
                        raise Violation("a wait without an arrival")
                    # a CTA that has ended counts as arrived
                    if any(x < a[c] and p < len(prog) for x, p in zip(arrived, pcs)):
                        continue
                    w[c] += 1
                elif op[0] == "store":
                    for d in range(ctas):
                        if d != c and pcs[d] == -1:
                            raise Violation(f"pass {op[1]}: a store into a CTA that has not started")
                        if d != c and pcs[d] == len(prog):
                            raise Violation(f"pass {op[1]}: a store into a CTA that has ended")
                    s = stored | {(c, op[1])}
                elif any((d, op[1]) not in stored for d in range(ctas)):
                    raise Violation(f"pass {op[1]}: read before every CTA has stored")
            moved = True
            n = (pcs[:c] + (pc + 1,) + pcs[c + 1:], tuple(a), tuple(w), s)
            if n not in seen:
                seen.add(n)
                todo.append(n)
        if not moved and any(p < len(prog) for p in pcs):
            raise Violation("some CTA waits forever")
    return len(seen)


@pytest.mark.parametrize("ctas", [2, 3, 4])
@pytest.mark.parametrize("passes", [1, 2])
def test_the_kernels_protocol(ctas, passes):
    prog = kernel_program(passes)
    assert [p for p in prog if p[0] == "store"] == [("store", k) for k in range(passes)]
    assert [p for p in prog if p[0] == "read"] == [("read", k) for k in range(passes)]
    assert check(prog, ctas) > 0


def test_a_missing_barrier_before_the_stores_is_caught():
    prog = kernel_program(2)
    assert prog[:2] == ["arrive", "wait"]
    with pytest.raises(Violation, match="has not started"):
        check(prog[2:], 2)


def test_a_missing_barrier_behind_the_stores_is_caught():
    prog = kernel_program(1)
    at = prog.index(("store", 0))
    assert prog[at + 1:at + 3] == ["arrive", "wait"]
    with pytest.raises(Violation, match="before every CTA has stored|has ended"):
        check(prog[:at + 1] + prog[at + 3:], 2)
