"""Chunk attention, draft verification, calibration and read-back on the CPU:
the library's refusals, the binding's checks, the block manager's runs of
tokens against a plain model of them, and the calls that PagedKVCache makes."""
import ctypes
import random

import numpy as np
import pytest
import torch

from paged_kv_cache_410_b200 import binding as B
from paged_kv_cache_410_b200.block_manager import (ERR_INVALID, ERR_NO_BLOCKS, BlockManager,
                                                   BlockManagerError)
from paged_kv_cache_410_b200.kv_cache import PagedKVCache

P = ctypes.c_void_p(1 << 20)      # an aligned address that is never followed
OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = range(5)


@pytest.fixture(scope="module")
def lib():
    return B.load_library()


def desc(**kw):
    d = dict(num_blocks=64, block_size=16, num_kv_heads=2, head_dim=64, cache_dtype=B.PA_F16,
             k_scale=None, v_scale=None, k_inv_scale=None, v_inv_scale=None)
    d.update(kw)
    return B._CacheDesc(*d.values())


def attend(lib, d=None, **kw):
    a = dict(q=P, dt=B.PA_F16, tokens=8, batch=2, hq=4, k=P, v=P, cu=P, most=4, tab=P, mb=4,
             lens=P, ctx=64, window=0, scale=0.125, out=P, part=0, ws=None, wsb=0)
    a.update(kw)
    d = d or desc()
    return lib.pa_attend_chunk(a["q"], a["dt"], a["tokens"], a["batch"], a["hq"], a["k"], a["v"],
                               ctypes.byref(d), a["cu"], a["most"], a["tab"], a["mb"], a["lens"],
                               a["ctx"], a["window"], a["scale"], a["out"], a["part"], a["ws"],
                               a["wsb"], None)


@pytest.mark.parametrize("change, want", [
    (dict(tokens=-1), INVALID), (dict(batch=-1), INVALID), (dict(hq=3), INVALID),
    (dict(hq=0), INVALID), (dict(most=-1), INVALID), (dict(window=-1), INVALID),
    (dict(dt=B.PA_E4M3), INVALID), (dict(dt=B.PA_F32), INVALID), (dict(dt=B.PA_BF16), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(cu=None), INVALID), (dict(tab=None), INVALID), (dict(lens=None), INVALID),
    (dict(out=None), INVALID), (dict(q=ctypes.c_void_p(8)), INVALID),
    (dict(out=ctypes.c_void_p(24)), INVALID), (dict(mb=0), INVALID), (dict(ctx=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(part=64), INVALID), (dict(part=200), INVALID), (dict(part=1 << 21), INVALID),
    (dict(batch=70000), UNSUPPORTED), (dict(ctx=(1 << 30) + 1), UNSUPPORTED),
    (dict(hq=2002), UNSUPPORTED),
    (dict(ctx=4096, part=128), WORKSPACE),                                   # none given
    (dict(ctx=4096, part=128, ws=P, wsb=100), WORKSPACE),                    # too small
    (dict(ctx=4096, part=128, ws=ctypes.c_void_p((1 << 20) + 16), wsb=1 << 30), WORKSPACE),
    (dict(batch=0), OK), (dict(tokens=0, q=None, out=None), OK), (dict(most=0), OK),
])
def test_attend_chunk_refusals(lib, change, want):
    assert attend(lib, **change) == want


def test_attend_chunk_cache_checks(lib):
    assert attend(lib, desc(block_size=12)) == INVALID
    assert attend(lib, desc(head_dim=96)) == UNSUPPORTED
    assert attend(lib, desc(cache_dtype=B.PA_F32)) == INVALID
    assert attend(lib, desc(cache_dtype=B.PA_E4M3)) == INVALID               # no scales


def test_attend_chunk_workspace_sizes(lib):
    def size(tokens=8, batch=2, hq=4, most=4, ctx=64, window=0, part=0, d=None):
        return lib.pa_attend_chunk_workspace_size(tokens, batch, hq, most, ctx, window, part,
                                                  ctypes.byref(d or desc()))
    assert size() == 0
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    rows = 8 * 4
    assert size(ctx=1000, part=128) == up(rows * 8 * 64 * 4) + up(rows * 8 * 8)
    # a window bounds the tokens a row tile sees, so the partitions too
    assert size(ctx=100000, window=100, part=128) <= up(rows * 3 * 64 * 4) + up(rows * 3 * 8)
    for bad in (dict(tokens=0), dict(batch=0), dict(hq=3), dict(most=0), dict(ctx=-1),
                dict(window=-1), dict(part=-1), dict(d=desc(block_size=12))):
        assert size(**dict(dict(ctx=100000), **bad)) == 0
    # as many rows as fill the GPU are not split; a few are
    many = desc(num_kv_heads=8, head_dim=128)
    assert size(tokens=512, batch=64, hq=64, most=8, ctx=4096, d=many) == 0
    assert size(tokens=5, batch=1, hq=64, most=5, ctx=100000, d=many) > 0


@pytest.mark.parametrize("change, want", [
    (dict(n=-1), INVALID), (dict(batch=-1), INVALID), (dict(vocab=0), INVALID),
    (dict(most=-1), INVALID), (dict(dt=B.PA_E4M3), INVALID), (dict(dt=7), INVALID),
    (dict(x=None), INVALID), (dict(cu=None), INVALID), (dict(p=None), INVALID),
    (dict(ua=None), INVALID), (dict(us=None), INVALID), (dict(acc=None), INVALID),
    (dict(tok=None), INVALID), (dict(p=ctypes.c_void_p(6)), INVALID),
    (dict(most=0x7fffffff), UNSUPPORTED), (dict(batch=0), OK),
])
def test_verify_refusals(lib, change, want):
    a = dict(x=P, n=6, batch=2, cu=P, p=P, q=P, dt=B.PA_F32, vocab=100, ua=P, us=P, most=3, acc=P,
             tok=P)
    a.update(change)
    assert lib.pa_verify_draft(a["x"], a["n"], a["batch"], a["cu"], a["p"], a["q"], a["dt"],
                               a["vocab"], a["ua"], a["us"], a["most"], a["acc"], a["tok"],
                               None) == want


@pytest.mark.parametrize("change", [
    dict(vocab=(1 << 30) + 1), dict(vocab=0x7fffffff), dict(most=(1 << 30) + 1)])
def test_verify_refuses_sizes_its_indices_do_not_hold(lib, change):
    a = dict(vocab=100, most=3)
    a.update(change)
    assert lib.pa_verify_draft(P, 6, 2, P, P, P, B.PA_F32, a["vocab"], P, P, a["most"], P, P,
                               None) == UNSUPPORTED


@pytest.mark.parametrize("change, want", [
    (dict(t=-1), INVALID), (dict(h=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(dt=B.PA_F32), INVALID), (dict(k=None), INVALID), (dict(v=ctypes.c_void_p(8)), INVALID),
    (dict(arrays=[P] * 5 + [None]), INVALID), (dict(arrays=[ctypes.c_void_p(4)] + [P] * 5), INVALID),
    (dict(h=70000), UNSUPPORTED),
])
def test_calibrate_refusals(lib, change, want):
    a = dict(k=P, v=P, dt=B.PA_F16, t=4, h=2, d=64, slots=None, arrays=[P] * 6)
    a.update(change)
    assert lib.pa_calibrate_kv(a["k"], a["v"], a["dt"], a["t"], a["h"], a["d"], a["slots"],
                               *a["arrays"], None) == want


@pytest.mark.parametrize("change, want", [
    (dict(mb=0), INVALID), (dict(batch=-1), INVALID), (dict(t=-1), INVALID),
    (dict(dt=B.PA_E4M3), INVALID), (dict(dt=B.PA_BF16), UNSUPPORTED), (dict(k=None), INVALID),
    (dict(tab=None), INVALID), (dict(first=None), INVALID), (dict(cu=None), INVALID),
    (dict(ko=ctypes.c_void_p(8)), INVALID), (dict(batch=0), OK), (dict(t=0, ko=None, vo=None), OK),
])
def test_gather_refusals(lib, change, want):
    a = dict(k=P, v=P, tab=P, mb=4, batch=2, first=P, cu=P, t=9, ko=P, vo=P, dt=B.PA_F16)
    a.update(change)
    d = desc()
    assert lib.pa_gather_kv(a["k"], a["v"], ctypes.byref(d), a["tab"], a["mb"], a["batch"],
                            a["first"], a["cu"], a["t"], a["ko"], a["vo"], a["dt"], None) == want
    d8 = desc(cache_dtype=B.PA_E4M3)
    if want == OK and a["batch"] and a["t"]:
        assert lib.pa_gather_kv(a["k"], a["v"], ctypes.byref(d8), a["tab"], a["mb"], a["batch"],
                                a["first"], a["cu"], a["t"], a["ko"], a["vo"], a["dt"], None) == INVALID


class Recorder:
    """Stands in for the CUDA entry points; the block manager stays the real one."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.startswith("pa_bm_"):
            return getattr(_real, name)

        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


_real = B.load_library()


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(B, "load_library", lambda *a, **k: r)
    monkeypatch.setattr(B, "_on_device", lambda t: True)
    return r


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_checks(rec):
    k = torch.zeros((8, 16, 2, 64), dtype=torch.float16)
    cache = B.PagedCache.for_tensor(k)
    q = torch.zeros((5, 4, 64), dtype=torch.float16)

    def call(**kw):
        a = dict(q=q, k_cache=k, v_cache=k, cu_chunk=i32(3), block_tables=i32(2, 4),
                 context_lens=i32(2), scale=1.0, out=torch.zeros_like(q), cache=cache, max_chunk=3,
                 max_context=20, stream=0)
        a.update(kw)
        B.pa_attend_chunk(**a)

    call()
    name, a = rec.calls[-1]
    assert name == "pa_attend_chunk" and a[2] == 5 and a[3] == 2 and a[4] == 4 and a[9] == 3
    for bad in (dict(cu_chunk=i32(2)), dict(cu_chunk=i32(3).long()), dict(context_lens=i32(3)),
                dict(q=q[:, :, :32]), dict(out=q[:4]), dict(out=q.float()), dict(q=q.float()),
                dict(block_tables=i32(2)), dict(k_cache=k[:4]), dict(q=q[0])):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    x, p = i32(3), torch.zeros((5, 100))
    u, us = torch.zeros(3), torch.zeros(2)

    def verify(**kw):
        a = dict(draft_tokens=x, cu_drafts=i32(3), target_probs=p, draft_probs=p[:3],
                 accept_uniforms=u, sample_uniforms=us, accepted=i32(2), tokens=i32(2, 4), stream=0)
        a.update(kw)
        B.pa_verify_draft(**a)

    verify()
    verify(draft_probs=None)
    assert rec.calls[-1][1][5] is None and rec.calls[-1][1][6] == B.PA_F32
    for bad in (dict(target_probs=p[:4]), dict(draft_probs=p), dict(draft_probs=p[:3].half()),
                dict(accept_uniforms=us), dict(sample_uniforms=u), dict(tokens=i32(3, 4)),
                dict(tokens=i32(2, 0)), dict(cu_drafts=i32(2)), dict(draft_tokens=x.long()),
                dict(target_probs=p.double())):
        with pytest.raises((ValueError, TypeError)):
            verify(**bad)
    kk, f = torch.zeros((3, 2, 64), dtype=torch.float16), torch.zeros((2, 64))
    B.pa_calibrate_kv(kk, kk, None, f, f, f, f, f, f, stream=0)
    with pytest.raises(ValueError):
        B.pa_calibrate_kv(kk, kk[:2], None, f, f, f, f, f, f, stream=0)
    with pytest.raises(TypeError):
        B.pa_calibrate_kv(kk, kk, None, f.double(), f, f, f, f, f, stream=0)
    B.pa_gather_kv(k, k, i32(2, 4), i32(2), i32(3), kk, kk, cache, stream=0)
    with pytest.raises(ValueError):
        B.pa_gather_kv(k, k, i32(2, 4), i32(3), i32(3), kk, kk, cache, stream=0)
    with pytest.raises(TypeError):
        B.pa_gather_kv(k, k, i32(2, 4), i32(2), i32(3), kk, kk.bfloat16(), cache, stream=0)


def test_tensors_of_another_device_are_refused(monkeypatch):
    class Fake:
        def __init__(self, at):
            self.at = at

        def get_device(self):
            return self.at

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    B._on_current(Fake(0), None, Fake(0))
    for bad in ((Fake(1), Fake(1)), (Fake(0), Fake(1))):
        with pytest.raises(ValueError):
            B._on_current(*bad)


def test_scales_of_another_device_are_refused(rec, monkeypatch):
    """The kernels read the cache's scales: they are among the tensors whose device is checked."""
    ones = torch.ones((2, 64))
    k = torch.zeros((8, 16, 2, 64), dtype=torch.uint8)
    cache = B.PagedCache.for_tensor(k, k_scale=ones, v_scale=ones.clone(), k_inv_scale=ones,
                                    v_inv_scale=ones)
    q, kk = torch.zeros((5, 4, 64), dtype=torch.float16), torch.zeros((5, 2, 64), dtype=torch.float16)
    for bad in (cache.k_scale, cache.v_scale):
        class Elsewhere(torch.Tensor):
            def get_device(self):
                return 1

        kw = {n: (t.as_subclass(Elsewhere) if t is bad else t) for n, t in
              (("k_scale", cache.k_scale), ("v_scale", cache.v_scale))}
        other = B.PagedCache.for_tensor(k, k_inv_scale=ones, v_inv_scale=ones, **kw)
        with pytest.raises(ValueError, match="device"):
            B.pa_attend_chunk(q, k, k, i32(3), i32(2, 4), i32(2), 1.0, torch.zeros_like(q), other, 3,
                              20, stream=0)
        with pytest.raises(ValueError, match="device"):
            B.pa_gather_kv(k, k, i32(2, 4), i32(2), i32(3), kk, kk, other, stream=0)
    B.pa_gather_kv(k, k, i32(2, 4), i32(2), i32(3), kk, kk, cache, stream=0)


# ---- block manager -------------------------------------------------------------
def test_chunks_equal_single_appends():
    a, b = BlockManager(64, 4, True), BlockManager(64, 4, True)
    for bm in (a, b):
        bm.add_sequence(1, list(range(6)))
        bm.add_sequence(2, list(range(9)))
        bm.fork(1, 3)
    lists = [[10, 11, 12, 13, 14], [], [20, 21]]
    slots, pairs = a.append_chunks([1, 2, 3], lists)
    assert len(slots) == 7 and len(pairs) == 1
    for s, toks in zip((1, 2, 3), lists):
        for t in toks:
            b.append_token(s, t)
    for s in (1, 2, 3):
        assert a.length(s) == b.length(s)
        n = a.length(s)
        assert len(set(a.slots(s, 0, n).tolist())) == n
    got = np.concatenate([a.slots(1, 6, 5), a.slots(3, 6, 2)])
    assert slots.tolist() == got.tolist()
    assert a.num_free_blocks == b.num_free_blocks


def test_chunks_fail_whole():
    bm = BlockManager(4, 4, False)
    bm.add_sequence(1, [1, 2, 3])
    bm.add_sequence(2, [1])
    before = bm.num_free_blocks, bm.length(1), bm.length(2)
    for ids, lists, code in (([1, 2], [[1] * 9, [1] * 4], ERR_NO_BLOCKS), ([1, 7], [[1], [1]], ERR_INVALID),
                             ([1, 1], [[1], [1]], ERR_INVALID)):
        with pytest.raises(BlockManagerError) as e:
            bm.append_chunks(ids, lists)
        assert e.value.code == code
        assert (bm.num_free_blocks, bm.length(1), bm.length(2)) == before
    for ids, lens in (([1], [4]), ([1, 1], [1, 1]), ([9], [0]), ([1], [-1])):
        with pytest.raises(BlockManagerError):
            bm.keep(ids, lens)
    bm.append_chunks([1, 2], [[1] * 5, [1] * 3])
    bm.release_before(1, 5)
    with pytest.raises(BlockManagerError):
        bm.keep([1], [3])                     # inside a released block
    bm.keep([1], [5])


@pytest.mark.parametrize("seed", range(8))
def test_drafts_kept_and_dropped_at_random(seed):
    """Random speculative steps, forks and new prompts: every sequence's tokens stay those of a
    plain model, no block serves two different contents, refused drafts never come back from the
    prefix cache, and every block returns in the end."""
    rng = random.Random(seed)
    bs, nb = 4, 400
    bm = BlockManager(nb, bs, True)
    model, cells, nxt = {}, {}, 0            # tokens; content of each slot

    def store(slots, ids):
        for s, t in zip(slots, ids):
            cells[int(s)] = t

    def check(sid):
        toks = model[sid]
        assert bm.length(sid) == len(toks)
        for j, s in enumerate(bm.slots(sid, 0, len(toks))):
            assert cells[int(s)] == tuple(toks[:j + 1]), (sid, j)

    def copy(pairs):
        for s, d in pairs:
            for r in range(bs):
                if s * bs + r in cells:
                    cells[d * bs + r] = cells[s * bs + r]

    def prefixes(toks, first):
        return [tuple(toks[:j + 1]) for j in range(first, len(toks))]

    for step in range(60):
        what = rng.random()
        if what < 0.2 or not model:
            toks = [rng.randint(0, 2) for _ in range(rng.randint(1, 14))]
            cached = bm.add_sequence(nxt, toks)
            model[nxt] = toks
            store(bm.slots(nxt, cached, len(toks) - cached), prefixes(toks, cached))
            check(nxt)
            nxt += 1
        elif what < 0.3:
            sid = rng.choice(list(model))
            bm.fork(sid, nxt)
            model[nxt] = list(model[sid])
            nxt += 1
        elif what < 0.4 and len(model) > 1:
            sid = rng.choice(list(model))
            bm.free_sequence(sid)
            del model[sid]
        else:
            ids = rng.sample(list(model), rng.randint(1, len(model)))
            drafts = rng.random() < 0.7
            lists = [[rng.randint(0, 2) for _ in range(rng.randint(1, 9))] for _ in ids]
            slots, pairs = bm.append_chunks(ids, lists, offer=not drafts)
            copy(pairs)
            at = 0
            for sid, run in zip(ids, lists):
                old = len(model[sid])
                model[sid] += run
                store(slots[at:at + len(run)], prefixes(model[sid], old))
                at += len(run)
            for sid in ids:
                check(sid)
            if drafts:
                keep = [len(model[s]) - rng.randint(0, len(r) - 1) for s, r in zip(ids, lists)]
                bm.keep(ids, keep)
                for sid, n in zip(ids, keep):
                    del model[sid][n:]
        for sid in model:
            check(sid)
    for sid in list(model):
        bm.free_sequence(sid)
    assert bm.num_free_blocks + bm.num_cached_blocks == nb


@pytest.mark.parametrize("how", ["chunks", "tokens"])
def test_a_copy_source_is_not_handed_out_in_its_batch(how):
    """Sequences cut inside a cached block copy it on the next append; the first one's source is
    then held by the cache alone, and the pool has no other block for the second one's copy but
    the one the third sequence left."""
    bm = BlockManager(4, 4, True)
    for sid in (1, 2, 3):
        bm.add_sequence(sid, [])
        bm.append_chunks([sid], [[10 * sid + i for i in range(4)]])
    bm.free_sequence(3)
    bm.keep([1, 2], [3, 3])
    old = [int(bm.slots(s, 0, 1)[0]) // 4 for s in (1, 2)]
    if how == "chunks":
        slots, pairs = bm.append_chunks([1, 2], [[40], [80]])
    else:
        slots, pairs = bm.append_tokens([1, 2], [40, 80])
    assert [p[0] for p in pairs.tolist()] == old and len({int(p[1]) for p in pairs}) == 2
    assert not {int(p[0]) for p in pairs} & {int(p[1]) for p in pairs}
    assert [int(s) // 4 for s in slots] == [int(p[1]) for p in pairs]
    # the sources are evictable again: the pool still serves two more blocks
    bm.free_sequence(2)
    bm.add_sequence(9, [1] * 12)


@pytest.mark.parametrize("how", ["chunks", "tokens"])
def test_sharers_of_a_held_block_still_write_in_place(how):
    """Three sequences share a partial block: two copy it, the last one writes in place."""
    bm = BlockManager(8, 4, True)
    bm.add_sequence(1, [1, 2])
    bm.fork(1, 2)
    bm.fork(1, 3)
    at = int(bm.slots(1, 0, 1)[0]) // 4
    slots, pairs = (bm.append_chunks([1, 2, 3], [[5], [6], [7]]) if how == "chunks"
                    else bm.append_tokens([1, 2, 3], [5, 6, 7]))
    assert len(pairs) == 2 and int(slots[2]) // 4 == at
    assert not {int(p[0]) for p in pairs} & {int(p[1]) for p in pairs}


@pytest.mark.parametrize("seed", range(12))
def test_keep_and_eviction_at_random(seed):
    """Random chunks, single steps, cuts, forks and new prompts in a pool that runs out: every
    sequence's tokens stay those of a plain model, the copies of a batch are applied all at once
    (no block is a source of one and the destination of another), and a refused call changes
    nothing."""
    rng = random.Random(seed)
    bs, nb = 4, 14
    bm = BlockManager(nb, bs, True)
    model, cells, nxt, copies, refused = {}, {}, 0, 0, 0

    def check():
        for sid, toks in model.items():
            assert bm.length(sid) == len(toks)
            for j, s in enumerate(bm.slots(sid, 0, len(toks))):
                assert cells[int(s)] == tuple(toks[:j + 1]), (sid, j)

    for step in range(300):
        what = rng.random()
        if what < 0.2 or not model:
            toks = [rng.randint(0, 1) for _ in range(rng.randint(1, 9))]
            try:
                cached = bm.add_sequence(nxt, toks)
            except BlockManagerError as e:
                assert e.code == ERR_NO_BLOCKS
                refused += 1
                if model:
                    sid = rng.choice(list(model))
                    bm.free_sequence(sid)
                    del model[sid]
                continue
            model[nxt] = toks
            for j, s in enumerate(bm.slots(nxt, cached, len(toks) - cached)):
                cells[int(s)] = tuple(toks[:cached + j + 1])
            nxt += 1
        elif what < 0.28:
            sid = rng.choice(list(model))
            bm.fork(sid, nxt)
            model[nxt] = list(model[sid])
            nxt += 1
        elif what < 0.4:
            sid = rng.choice(list(model))
            bm.free_sequence(sid)
            del model[sid]
        elif what < 0.6:
            ids = rng.sample(list(model), rng.randint(1, len(model)))
            keep = [rng.randint(max(0, len(model[s]) - 5), len(model[s])) for s in ids]
            bm.keep(ids, keep)
            for s, n in zip(ids, keep):
                del model[s][n:]
        else:
            ids = rng.sample(list(model), rng.randint(1, len(model)))
            single = rng.random() < 0.4
            lists = [[rng.randint(0, 1) for _ in range(1 if single else rng.randint(0, 5))]
                     for _ in ids]
            try:
                if single:
                    slots, pairs = bm.append_tokens(ids, [r[0] for r in lists])
                else:
                    slots, pairs = bm.append_chunks(ids, lists, offer=rng.random() < 0.5)
            except BlockManagerError as e:
                assert e.code == ERR_NO_BLOCKS
                refused += 1
                check()
                continue
            copies += len(pairs)
            dst = [int(p[1]) for p in pairs]
            assert len(set(dst)) == len(dst) and not set(dst) & {int(p[0]) for p in pairs}
            for s, d in pairs:
                for r in range(bs):
                    if s * bs + r in cells:
                        cells[int(d) * bs + r] = cells[int(s) * bs + r]
            at = 0
            for sid, run in zip(ids, lists):
                for t in run:
                    model[sid].append(t)
                    cells[int(slots[at])] = tuple(model[sid])
                    at += 1
        check()
    assert copies > 0 and refused > 0
    for sid in list(model):
        bm.free_sequence(sid)
    assert bm.num_free_blocks + bm.num_cached_blocks == nb


def test_refused_drafts_are_not_cached():
    bm = BlockManager(32, 4, True)
    bm.add_sequence(1, [1, 2, 3])
    bm.append_chunks([1], [[4, 5, 6, 7, 8]], offer=False)
    bm.keep([1], [4])
    assert bm.add_sequence(2, [1, 2, 3, 4, 5, 6, 7, 8, 9]) == 4


# ---- PagedKVCache ---------------------------------------------------------------
def test_chunk_plan_and_calls(rec):
    c = PagedKVCache(64, 4, 2, 64, num_layers=2, device="cpu", max_blocks_per_seq=16, stream=0)
    twin = BlockManager(64, 4, True)
    for sid, prompt in ((0, list(range(10))), (1, [5, 6])):
        c.add_sequence(sid, prompt)
        twin.add_sequence(sid, prompt)
    c.fork(0, 2)
    twin.fork(0, 2)
    rec.calls.clear()
    lists = [[7, 8, 9], [3], [1, 2]]
    plan = c.begin_chunk([0, 1, 2], lists, drafts=True)
    slots, pairs = twin.append_chunks([0, 1, 2], lists, offer=False)
    assert plan.slot_mapping.tolist() == slots.tolist() and plan.copy_pairs.tolist() == pairs.tolist()
    assert [n for n, _ in rec.calls] == ["pa_copy_blocks_layers"] and len(pairs) == 1
    tables, lens = twin.block_tables([0, 1, 2], 16)
    assert np.array_equal(plan.block_tables.numpy(), tables)
    assert plan.context_lens.tolist() == lens.tolist() == [13, 3, 12]
    assert plan.cu_chunk.tolist() == [0, 3, 4, 6] and plan.max_chunk == 3 and plan.max_context == 13
    assert plan.drafts.tolist() == [8, 9, 2] and plan.cu_drafts.tolist() == [0, 2, 2, 3]
    q, k = torch.zeros((6, 4, 64), dtype=torch.float16), torch.zeros((6, 2, 64), dtype=torch.float16)
    rec.calls.clear()
    out = c.attend_chunk(plan, 1, q, k, k)
    names = [n for n, _ in rec.calls]
    assert names == ["pa_append_kv", "pa_attend_chunk_workspace_size", "pa_attend_chunk"]
    a = rec.calls[-1][1]
    assert a[0] == q.data_ptr() and a[5] == c.k[1].data_ptr() and a[16] == out.data_ptr()
    p = torch.zeros((6, 50))
    acc, tok = c.verify(plan, p, p[:3], torch.zeros(3), torch.zeros(3))
    assert rec.calls[-1][0] == "pa_verify_draft" and tuple(tok.shape) == (3, 3) and len(acc) == 3
    with pytest.raises(ValueError):
        c.settle(plan, [3, 0, 0])                # more than were drafted
    c.settle(plan, torch.tensor([1, 0, 0], dtype=torch.int32))
    assert [c.bm.length(s) for s in (0, 1, 2)] == [12, 3, 11]
    plain = c.begin_chunk([1], [[4, 4]])
    for bad in (lambda: c.settle(plain, [0]), lambda: c.verify(plain, p, None, p, p),
                lambda: c.begin_chunk([0, 1], [[1]]), lambda: c.begin_chunk([0], [[]], drafts=True),
                lambda: c.begin_chunk([0], [[1] * 100])):
        with pytest.raises(ValueError):
            bad()
    assert [c.bm.length(s) for s in (0, 1, 2)] == [12, 5, 11]


def test_plan_of_a_placed_prompt(rec):
    c = PagedKVCache(64, 4, 2, 64, device="cpu", max_blocks_per_seq=16, stream=0)
    assert c.add_sequence(0, list(range(10)))[0] == 0
    cached, slots = c.add_sequence(1, list(range(8)) + [50, 51, 52])
    assert cached == 8
    plan = c.plan_chunk([1], [cached])
    assert plan.slot_mapping.tolist() == slots.tolist() and plan.counts.tolist() == [3]
    assert plan.context_lens.tolist() == [11] and plan.max_context == 11 and plan.max_chunk == 3
    assert plan.cu_chunk.tolist() == [0, 3] and plan.drafts is None and len(plan.copy_pairs) == 0
    assert np.array_equal(plan.block_tables.numpy(), c.bm.block_tables([1], 16)[0])
    # pieces, beside another sequence's; nothing is reserved by a plan
    plan = c.plan_chunk([0, 1], [0, 9], [6, 1])
    assert plan.slot_mapping.tolist() == c.bm.slots(0, 0, 6).tolist() + c.bm.slots(1, 9, 1).tolist()
    assert plan.context_lens.tolist() == [6, 10] and plan.cu_chunk.tolist() == [0, 6, 7]
    assert [c.bm.length(s) for s in (0, 1)] == [10, 11]
    # a prompt cached whole: its last row, whose K/V is not stored again
    assert c.add_sequence(2, list(range(8)))[0] == 8
    plan = c.plan_chunk([2, 0], [7, 6], stored=[8, 8])
    assert plan.slot_mapping.tolist() == [-1, -1, -1] + c.bm.slots(0, 8, 2).tolist()
    assert plan.context_lens.tolist() == [8, 10]
    q, k = torch.zeros((5, 4, 64), dtype=torch.float16), torch.zeros((5, 2, 64), dtype=torch.float16)
    rec.calls.clear()
    c.attend_chunk(plan, 0, q, k, k)
    assert [n for n, _ in rec.calls] == ["pa_append_kv", "pa_attend_chunk_workspace_size",
                                         "pa_attend_chunk"]
    for bad in (([0], [-1]), ([0], [11]), ([0], [5], [6]), ([0], [5], [-1]), ([0, 1], [5]),
                ([0], [5], [1, 1]), ([0], [5], [1], [1, 2])):
        with pytest.raises(ValueError):
            c.plan_chunk(*bad)
    with pytest.raises(BlockManagerError):
        c.plan_chunk([77], [0])
    assert c.plan_chunk([], []).cu_chunk.tolist() == [0]
    assert c.plan_chunk([0], [10]).counts.tolist() == [0]


def test_plan_of_a_placed_prompt_with_a_window(rec):
    c = PagedKVCache(64, 4, 2, 64, device="cpu", max_blocks_per_seq=32, stream=0, window=6)
    c.add_sequence(0, list(range(30)))
    before = c.plan_chunk([0], [0], [20]).block_tables.clone()
    assert len(c.bm.slots(0, 0, 30)) == 30
    plan = c.plan_chunk([0], [20])                # its first row sees 15 .. 20
    assert torch.equal(plan.block_tables, before)
    assert len(c.bm.slots(0, 12, 18)) == 18
    with pytest.raises(BlockManagerError):
        c.plan_chunk([0], [11])


def test_read_and_calibrate_calls(rec):
    ones = [torch.ones((2, 64))]
    c = PagedKVCache(64, 4, 2, 64, dtype=torch.uint8, io_dtype=torch.float16, device="cpu",
                     max_blocks_per_seq=16, stream=0, k_scales=ones, v_scales=ones)
    c.add_sequence(0, list(range(10)))
    k, v = c.read(0, 0, 2, 5)
    assert tuple(k.shape) == (5, 2, 64) and k.dtype == torch.float16
    assert rec.calls[-1][0] == "pa_gather_kv" and rec.calls[-1][1][8] == 5
    assert c.read(0, 0)[0].shape[0] == 10
    for first, count in ((-1, 2), (0, 11), (8, 3), (4, -1)):
        with pytest.raises(ValueError):
            c.read(0, 0, first, count)
    x = torch.zeros((3, 2, 64), dtype=torch.float16)
    c.calibrate(0, x, x)
    c.calibrate(0, x, x)
    a, b = (args for n, args in rec.calls if n == "pa_calibrate_kv")
    assert a[7:] == b[7:] and a[9] == c.layers[0].k_scale.data_ptr()
    assert bool((ones[0] == 1).all())              # the caller's scales are not written
    plain = PagedKVCache(8, 4, 2, 64, device="cpu", stream=0)
    with pytest.raises(ValueError):
        plain.calibrate(0, x, x)


def test_a_refused_calibration_leaves_the_scales(rec):
    twos = [torch.full((2, 64), 2.0)]
    c = PagedKVCache(64, 4, 2, 64, dtype=torch.uint8, io_dtype=torch.float16, device="cpu",
                     max_blocks_per_seq=16, stream=0, k_scales=twos, v_scales=twos)
    x = torch.zeros((3, 2, 64), dtype=torch.float16)
    bad = [(x[:, :1], x, None), (x, x[:2], None), (x.float(), x, None), (x, x.bfloat16(), None),
           (x.transpose(1, 2), x, None), (x, x, i32(3)), (x, x, torch.zeros(2, dtype=torch.int64))]
    layer = c.layers[0]

    def scales():
        return layer.k_scale, layer.v_scale, layer.k_inv_scale, layer.v_inv_scale

    before = scales()
    for args in bad:
        with pytest.raises((ValueError, TypeError)):
            c.calibrate(0, *args)
        assert all(a is b for a, b in zip(scales(), before)) and c._amax[0] is None
    assert bool((layer.k_scale == 2).all()) and bool((layer.k_inv_scale == 0.5).all())
    c.calibrate(0, x, x)                          # the stub leaves zeros: new arrays are in place
    after = scales()
    assert all(a is not b for a, b in zip(after, before))
    for args in bad:
        with pytest.raises((ValueError, TypeError)):
            c.calibrate(0, *args)
        assert all(a is b for a, b in zip(scales(), after))


def test_window_releases_only_what_no_new_token_sees(rec):
    c = PagedKVCache(64, 4, 2, 64, device="cpu", max_blocks_per_seq=32, stream=0, window=6)
    c.add_sequence(0, list(range(20)))
    c.begin_chunk([0], [[1, 2, 3]])               # rows at 20..22: the first sees 15..20
    assert len(c.bm.slots(0, 12, 11)) == 11       # block 3 (tokens 12..15) is still held
    with pytest.raises(BlockManagerError):
        c.bm.slots(0, 11, 1)
