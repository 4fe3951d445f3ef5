"""The ring of K and V buffers of the chunk kernel
(paged_kv_cache_410_b200/csrc/pa_chunk.cuh), model-checked on the CPU for one
row tile.

The roles: two TMA producers (K(it) is use 2 it of the ring, V(it) use
2 it + 1), a warp that issues S(it) = Q K(it)^T, one that issues P.V(it), and
the softmax warps between them. Copies land, and MMAs complete, in any
order that hardware may take (MMAs of one warp in order), and the arrivals
of an MMA's two commits on their barriers come apart and in any order. A
barrier counts its completed phases; a parity wait sees only whether the
phase before the current one has the named parity. The checks:

  * no parity wait that fires for a phase that has not completed;
  * no buffer loaded before the use before it has been read;
  * no state where some role waits forever.

`bars` is the number of barriers that the ring's uses are spread over: the
kernel's rule is read from its source.
"""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "paged_kv_cache_410_b200", "csrc", "pa_chunk.cuh")


class Violation(Exception):
    pass


def kernel_bars(bufs):
    with open(SOURCE) as f:
        m = re.search(r"kBars = kBufs % 2 \? (\d) \* kBufs : kBufs;", f.read())
    return int(m.group(1)) * bufs if bufs % 2 else bufs


def check(nsteps, bufs, bars, ask_ahead=True, limit=4000000):
    """Explore every interleaving (depth first); returns the number of states."""
    FULL, FREE, S, P, PV = 0, bars, 2 * bars, 2 * bars + 2, 2 * bars + 4

    def fired(bar, index, k, what):
        c = bar[index]
        if (c & 1) == (k & 1):
            return False
        if c <= k:
            raise Violation(f"{what}: fired for phase {k} with {c} completed")
        return True

    # state: producers' next steps, S / P.V / softmax positions, copies in
    # flight, MMAs issued and not complete (in order per kind), arrivals due,
    # uses read so far, barriers' completed phases
    start = ((0, 0), 0, 0, 0, frozenset(), (), (), frozenset(), frozenset(), (0,) * (2 * bars + 6))
    seen, todo = {start}, [start]
    while todo:
        st = todo.pop()
        prod, s, pv, sm, flying, s_ops, pv_ops, due, read, bar = st
        out = []

        def bump(b, index):
            return b[:index] + (b[index] + 1,) + b[index + 1:]

        for kv in (0, 1):                                          # ---- producers
            it = prod[kv]
            n = 2 * it + kv
            if it < nsteps and (n < bufs or fired(bar, FREE + (n - bufs) % bars,
                                                  (n - bufs) // bars, f"load {n}")):
                if n >= bufs and n - bufs not in read:
                    raise Violation(f"use {n} loaded before use {n - bufs} was read")
                out.append(((prod[0] + (kv == 0), prod[1] + (kv == 1)), s, pv, sm, flying | {n},
                            s_ops, pv_ops, due, read, bar))
        for n in flying:                                           # ---- copies land
            out.append((prod, s, pv, sm, flying - {n}, s_ops, pv_ops, due, read,
                        bump(bar, FULL + n % bars)))
        if s < nsteps:                                             # ---- the S warp
            n = 2 * s
            free = [lambda: s < 2 or fired(bar, PV + (s & 1), (s - 2) >> 1, f"S({s}) P.V"),
                    lambda: fired(bar, FULL + n % bars, n // bars, f"S({s}) K")]
            if all(wait() for wait in (reversed(free) if ask_ahead else free)):
                out.append((prod, s + 1, pv, sm, flying, s_ops + (s,), pv_ops, due, read, bar))
        if pv < nsteps:                                            # ---- the P.V warp
            n = 2 * pv + 1
            early = ask_ahead and fired(bar, FULL + n % bars, n // bars, f"P.V({pv}) V")
            if fired(bar, P + (pv & 1), pv >> 1, f"P.V({pv}) P") and \
                    (early or fired(bar, FULL + n % bars, n // bars, f"P.V({pv}) V")):
                out.append((prod, s, pv + 1, sm, flying, s_ops, pv_ops + (pv,), due, read, bar))
        if sm < nsteps and fired(bar, S + (sm & 1), sm >> 1, f"softmax {sm}"):
            out.append((prod, s, pv, sm + 1, flying, s_ops, pv_ops, due, read,
                        bump(bar, P + (sm & 1))))                  # ---- softmax
        if s_ops:                                                  # ---- MMAs complete
            it = s_ops[0]
            out.append((prod, s, pv, sm, flying, s_ops[1:], pv_ops,
                        due | {(S + (it & 1), it), (FREE + 2 * it % bars, it)}, read | {2 * it}, bar))
        if pv_ops:
            it = pv_ops[0]
            out.append((prod, s, pv, sm, flying, s_ops, pv_ops[1:],
                        due | {(PV + (it & 1), it), (FREE + (2 * it + 1) % bars, it)},
                        read | {2 * it + 1}, bar))
        for d in due:                                              # ---- commits arrive
            if any(e[0] == d[0] and e[1] < d[1] for e in due):
                continue                                           # (of one barrier: in order)
            out.append((prod, s, pv, sm, flying, s_ops, pv_ops, due - {d}, read, bump(bar, d[0])))
        if not out and not (prod == (nsteps, nsteps) and s == pv == sm == nsteps and not due):
            raise Violation(f"waits forever: S {s}, P.V {pv}, softmax {sm}")
        for n in out:
            if n not in seen:
                seen.add(n)
                todo.append(n)
        if len(seen) > limit:
            raise AssertionError("more states than expected")
    return len(seen)


@pytest.mark.parametrize("bufs,nsteps", [(3, 4), (3, 10), (4, 9), (5, 11), (6, 9)])
def test_the_kernels_ring(bufs, nsteps):
    bars = kernel_bars(bufs)
    assert bars % 2 == 0
    assert check(nsteps, bufs, bars) > 0


@pytest.mark.parametrize("bufs", [3, 5])
def test_one_barrier_per_buffer_of_an_odd_ring_is_caught(bufs):
    """K and V share the buffers of an odd ring: each producer sees every second phase of a
    buffer's barrier only, and a late arrival lets it pass a phase early."""
    with pytest.raises(Violation, match="load .*fired for phase"):
        check(12, bufs, bufs, ask_ahead=False)


def test_asking_ahead_on_shared_barriers_is_caught():
    with pytest.raises(Violation, match="fired for phase"):
        check(8, 3, 3)
