"""The turns of the chunk kernel's two row tiles on the exponential unit
(paged_kv_cache_410_b200/csrc/pa_chunk.cuh), model-checked on the CPU.

Two warps hand each other turns through two named barriers of 64 threads (a
warp's bar.sync or bar.arrive brings 32; bar.sync waits until the barrier is
full). Every other wait of a warp has a limit, so a warp may give up before
any turn, or behind it. Whatever the two do, no warp may wait for good.

`give_up` is what a warp does then: "takes its turns" (the kernel: the rest
of its turns empty-handed) or "hands on once" (a form in which the other
looks at an abort flag before each of its turns, and a warp that gives up
arrives once more: the other may have looked already).
"""
import os

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "paged_kv_cache_410_b200", "csrc", "pa_chunk.cuh")


class Violation(Exception):
    pass


def check(turns, give_up):
    """Explore every interleaving; returns the number of states."""
    # a warp: (turn, place, gave up); places: start (tile 1 opens tile 0's
    # first turn), look, sync, wait (in bar.sync), hand, behind, last, end
    start = ((0, "look", False), (0, "start", False), (0, 0), False)
    seen, todo = {start}, [start]

    def arrive(bars, warps, b):
        """32 threads more on barrier b (the warp's own index); full: its waiter goes on."""
        n = list(bars)
        n[b] += 1
        w = list(warps)
        if n[b] == 2:
            n[b] = 0
            k, place, gone = w[b]
            if place == "wait":
                w[b] = (k, "hand", gone)
        return tuple(n), w

    while todo:
        st = todo.pop()
        warps, bars, abort = st[:2], st[2], st[3]
        out = []
        for i in (0, 1):
            k, place, gone = warps[i]
            w = list(warps)

            def go(place, k=k, gone=gone, bars=bars, w=w, abort=abort):
                w = list(w)
                w[i] = (k, place, gone)
                out.append((w[0], w[1], bars, abort))

            if place == "start":
                n, w2 = arrive(bars, warps, 0)
                go("look", bars=n, w=w2)
            elif place in ("look", "behind"):
                if place == "behind":
                    go("look", k=k + 1)
                    if not gone:                   # a bounded wait behind the turn fails
                        go("look" if give_up == "takes its turns" else "last", k=k + 1, gone=True,
                           abort=True)
                elif k == turns:
                    go("end")
                elif gone:
                    go("sync")
                elif give_up == "takes its turns":
                    go("sync")
                    go("sync", gone=True, abort=True)
                else:
                    go("last" if abort else "sync")  # the flag, read before the turn
                    go("last", gone=True, abort=True)
            elif place == "sync":
                w[i] = (k, "wait", gone)
                n, w2 = arrive(bars, w, i)
                out.append((w2[0], w2[1], n, abort))
            elif place == "hand":
                if i == 0 or k + 1 < turns:
                    n, w2 = arrive(bars, warps, 1 - i)
                    go("behind", bars=n, w=w2)
                else:
                    go("behind")
            elif place == "last":                  # "hands on once"
                n, w2 = arrive(bars, warps, 1 - i)
                go("end", bars=n, w=w2)
        if not out and any(w[1] != "end" for w in warps):
            raise Violation(f"a warp waits for good: {warps}")
        for n in out:
            if n not in seen:
                seen.add(n)
                todo.append(n)
    return len(seen)


@pytest.mark.parametrize("turns", [1, 2, 3, 6])
def test_a_warp_that_gives_up_takes_its_turns(turns):
    assert check(turns, "takes its turns") > 0
    with open(SOURCE) as f:
        assert "for (; next_turn < turn_b; ++next_turn)" in f.read()


def test_handing_on_once_can_strand_the_other():
    with pytest.raises(Violation, match="waits for good"):
        check(3, "hands on once")
