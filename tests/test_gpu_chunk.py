"""Chunk attention over the paged cache (pa_attend_chunk) on the GPU, against
float64 attention row by row (tests/chunk_plain.py, whose docstring derives
the bound that every value is held to)."""
import math

import pytest
import torch

from paged_kv_cache_410_b200 import binding as B
from chunk_plain import attend_chunk, chunk_case, on_gpu

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def cache_of(g):
    sc = {}
    if g["k"].dtype == torch.uint8:
        sc = dict(k_scale=g["k_scale"], v_scale=g["v_scale"], k_inv_scale=1 / g["k_scale"],
                  v_inv_scale=1 / g["v_scale"])
    return B.PagedCache.for_tensor(g["k"], **sc)


def call(g, window=0, partition_tokens=0, scale=None, stream=None, out=None, workspace="own"):
    cache = cache_of(g)
    need = B.pa_attend_chunk_workspace_size(g["q"].shape[0], g["tables"].shape[0],
                                            g["q"].shape[1], g["max_chunk"], g["max_context"],
                                            cache, window, partition_tokens)
    ws = workspace
    if ws == "own":
        ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda") if need else None
    out = g["out"].clone() if out is None else out
    B.pa_attend_chunk(g["q"], g["k"], g["v"], g["cu"], g["tables"], g["lens"],
                      g["scale"] if scale is None else scale, out, cache, g["max_chunk"],
                      g["max_context"], window=window, partition_tokens=partition_tokens,
                      workspace=ws, stream=stream)
    return out


def check(c, got, window=0, scale=None):
    want, bound = attend_chunk(c["q"], c["k"], c["v"], c["cu"], c["tables"], c["lens"],
                               c["scale"] if scale is None else scale, c["out"], window,
                               c["k_scale"], c["v_scale"])
    err = (got.cpu().double() - want).abs()
    assert bool(torch.isfinite(got).all())
    worst = float((err - bound).max())
    assert worst <= 0, f"error {float(err.max())} passes the bound by {worst}"


# (hq, hkv, d, bs, dtype, cache): head layouts, block sizes and types
LAYOUTS = [
    (8, 8, 64, 16, F16, "io"),
    (4, 4, 128, 16, BF16, "io"),
    (16, 2, 128, 16, BF16, "io"),
    (6, 2, 64, 32, F16, "io"),      # 3 heads per KV head: 126 of a tile's 128 rows
    (7, 1, 128, 8, BF16, "io"),
    (4, 2, 128, 64, F16, "io"),
    (4, 2, 64, 128, BF16, "io"),
    (2, 1, 128, 256, F16, "io"),
    (4, 2, 128, 4, F16, "io"),      # blocks too small for TMA boxes
    (2, 1, 64, 1, BF16, "io"),
    (8, 2, 128, 16, F16, "e4m3"),
    (4, 1, 64, 32, BF16, "e4m3"),
    (6, 2, 128, 2, F16, "e4m3"),
    (130, 1, 64, 16, F16, "io"),    # more heads per KV head than a tile has rows
]
# (chunks, contexts)
SHAPES = [
    ([1], [1]),
    ([3, 1, 5], [3, 70, 200]),
    ([0, 4, 0, 1], [9, 130, 0, 1]),
    ([40, 1, 0, 129], [300, 64, 5, 129]),
]


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_matches_float64(layout, shape):
    hq, hkv, d, bs, dtype, cache = layout
    chunks, ctxs = SHAPES[shape]
    c = chunk_case(len(chunks), hq, hkv, d, bs, dtype, chunks, ctxs, cache, pad=3, seed=shape)
    g = on_gpu(c)
    got = call(g)
    assert B.pa_get_device_error() == 0
    check(c, got)
    assert torch.equal(got[int(c["cu"][-1]):].cpu(), c["out"][int(c["cu"][-1]):])


@pytest.mark.parametrize("layout", [0, 2, 3, 8, 10, 11], ids=lambda i: str(LAYOUTS[i]))
@pytest.mark.parametrize("window", [1, 7, 64, 100, 1000])
@pytest.mark.parametrize("part", [0, 128])
def test_window(layout, window, part):
    hq, hkv, d, bs, dtype, cache = LAYOUTS[layout]
    chunks, ctxs = [5, 1, 150], [400, 33, 310]
    c = chunk_case(3, hq, hkv, d, bs, dtype, chunks, ctxs, cache, pad=1, seed=window)
    # blocks the first row's window has left behind: freed, their entries anything
    for b in range(3):
        gone = max(0, ctxs[b] - chunks[b] - window + 1) // bs
        for i in range(gone):
            blk = int(c["tables"][b, i])
            if cache == "e4m3":
                c["k"][blk] = 0x7f
                c["v"][blk] = 0x7f
            else:
                c["k"][blk] = float("nan")
                c["v"][blk] = float("nan")
    plain = dict(c)
    plain["k"], plain["v"] = c["k"].clone(), c["v"].clone()
    g = on_gpu(c)
    for b in range(3):
        gone = max(0, ctxs[b] - chunks[b] - window + 1) // bs
        g["tables"][b, :gone] = -5
    got = call(g, window=window, partition_tokens=part)
    assert B.pa_get_device_error() == 0
    check(plain, got, window)


@pytest.mark.parametrize("layout", [1, 2, 5, 8, 10], ids=lambda i: str(LAYOUTS[i]))
@pytest.mark.parametrize("part", [128, 256, 1024])
def test_split_contexts(layout, part):
    hq, hkv, d, bs, dtype, cache = LAYOUTS[layout]
    c = chunk_case(3, hq, hkv, d, bs, dtype, [2, 70, 1], [700, 641, 1], cache, pad=2, seed=part)
    got = call(on_gpu(c), partition_tokens=part)
    assert B.pa_get_device_error() == 0
    check(c, got)


def test_many_sequences():
    """More sequences than one probe of the tile search covers, with empty ones among them."""
    n = 1100
    chunks = [(i * 7) % 4 for i in range(n)]
    ctxs = [c + (i % 40) for i, c in enumerate(chunks)]
    c = chunk_case(n, 2, 1, 64, 16, F16, chunks, ctxs, pad=1)
    got = call(on_gpu(c))
    assert B.pa_get_device_error() == 0
    check(c, got)


@pytest.mark.parametrize("window", [0, 50, 2 ** 31 - 1])
def test_longest_first(window):
    """More one-tile CTAs than the GPU holds: visited by context length, equal ones by index."""
    chunks = [(i * 3) % 5 for i in range(45)]
    ctxs = [c + [0, 7, 7, 100, 64, 3][i % 6] for i, c in enumerate(chunks)]
    c = chunk_case(45, 8, 8, 64, 16, F16, chunks, ctxs, pad=2)
    got = call(on_gpu(c), window=window)
    assert B.pa_get_device_error() == 0
    check(c, got, min(window, 1000))
    # the same with chunks longer than a row tile (two-tile CTAs)
    c = chunk_case(3, 2, 1, 64, 16, BF16, [70, 1, 140], [70, 90, 150])
    check(c, call(on_gpu(c), window=window), min(window, 1000))


@pytest.mark.parametrize("cache", ["io", "e4m3"])
@pytest.mark.parametrize("window", [0, 30])
def test_mixed_batch_of_many(cache, window):
    """Chunks longer than a row tile among many single tokens and empty chunks: two launches."""
    chunks = [140 if i in (3, 38) else 70 if i == 17 else (i % 4 != 1) * 1 for i in range(40)]
    ctxs = [c + (i * 13) % 90 for i, c in enumerate(chunks)]
    c = chunk_case(40, 16, 8, 64, 16, F16, chunks, ctxs, cache, pad=2)
    g = on_gpu(c)
    got = call(g, window=window)
    # work enqueued behind the call sees both launches' results
    copy = call(g, window=window).clone()
    assert B.pa_get_device_error() == 0
    check(c, got, window)
    assert torch.equal(got, copy)
    assert torch.equal(got[-2:].cpu(), c["out"][-2:])


def test_in_place():
    """The result may overwrite the queries."""
    c = chunk_case(2, 8, 2, 128, 16, BF16, [50, 3], [120, 400])
    g = on_gpu(c)
    want = call(g)
    q = g["q"].clone()
    assert torch.equal(call(dict(g, q=q), out=q), want)


@pytest.mark.parametrize("scale", [-0.125, 0.0, 3.0, 1e-6])
def test_scales(scale):
    c = chunk_case(2, 4, 2, 64, 16, F16, [9, 2], [50, 150])
    got = call(on_gpu(c), scale=scale)
    check(c, got, scale=scale)


def test_infinite_keys_of_later_tokens():
    """K of tokens a row does not see never reaches it, whatever its bits."""
    c = chunk_case(1, 2, 1, 128, 16, BF16, [20], [90])
    blk, row = int(c["tables"][0, 89 // 16]), 89 % 16
    k = c["k"].clone()
    k[blk, row] = float("inf")
    g = on_gpu(dict(c, k=k))
    got = call(g)
    want, bound = attend_chunk(c["q"], c["k"], c["v"], c["cu"], c["tables"], c["lens"], c["scale"],
                               c["out"])
    err = (got.cpu().double() - want).abs()[:19]
    assert bool((err <= bound[:19]).all())


def test_one_token_chunks_agree_with_decode():
    c = chunk_case(5, 8, 2, 128, 16, F16, [1] * 5, [1, 16, 17, 200, 333], junk=False)
    g = on_gpu(c)
    got = call(g)
    out = torch.empty_like(got)
    cache = cache_of(g)
    need = B.pa_decode_workspace_size(5, 8, 333, cache)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    B.pa_decode(g["q"], g["k"], g["v"], g["tables"], g["lens"], c["scale"], out, cache, 333,
                workspace=ws)
    check(c, out)
    check(c, got)


def test_repeats_bit_for_bit_and_on_another_stream():
    c = chunk_case(3, 8, 1, 128, 16, BF16, [33, 1, 6], [500, 64, 1000])
    g = on_gpu(c)
    a = call(g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = g["out"].clone()
    torch.cuda.synchronize()
    call(g, stream=s, out=b)
    s.synchronize()
    assert torch.equal(a, b)
    assert torch.equal(a, call(g))


@pytest.mark.parametrize("cache", ["io", "e4m3"])
def test_captured_and_replayed_with_new_inputs(cache):
    c = chunk_case(2, 8, 2, 128, 16, F16, [4, 3], [900, 333], cache)
    g = on_gpu(c)
    cc = cache_of(g)
    need = B.pa_attend_chunk_workspace_size(7, 2, 8, 4, 900, cc, 0, 128)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = g["out"].clone()
    call(g, partition_tokens=128, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(g, partition_tokens=128, out=out, workspace=ws, stream=torch.cuda.current_stream())
    # other queries, other lengths of the same launch
    c2 = dict(c, q=torch.randn(c["q"].shape, generator=torch.Generator().manual_seed(5)).to(F16),
              cu=torch.tensor([0, 1, 4], dtype=torch.int32),
              lens=torch.tensor([700, 128], dtype=torch.int32))
    g["q"].copy_(c2["q"])
    g["cu"].copy_(c2["cu"])
    g["lens"].copy_(c2["lens"])
    out.copy_(c["out"])
    graph.replay()
    torch.cuda.synchronize()
    assert B.pa_get_device_error() == 0
    check(c2, out)


def test_device_bounds_are_reported_not_faulted():
    c = chunk_case(3, 4, 2, 64, 16, F16, [2, 3, 4], [40, 50, 60], pad=1)
    def run(**change):
        g = on_gpu(dict(c, **{k: v for k, v in change.items()}))
        out = call(g)
        return out.cpu(), B.pa_get_device_error()

    ok, err = run()
    assert err == 0
    # a length shorter than its chunk, past max_context: zero rows, the others as before
    for bad in (2, 61):
        lens = torch.tensor([40, bad, 60], dtype=torch.int32)
        g = on_gpu(dict(c, lens=lens))
        out = call(g)
        assert B.pa_get_device_error() == B.DEVERR_CONTEXT_LEN
        assert bool((out[2:5] == 0).all())
        assert torch.equal(out[:2].cpu(), ok[:2]) and torch.equal(out[5:].cpu(), ok[5:])
    # a block id out of range
    t = c["tables"].clone()
    t[0, 1] = c["k"].shape[0]
    out, err = run(tables=t)
    assert err == B.DEVERR_BLOCK_ID and torch.equal(out[2:], ok[2:])
    # row starts that run backwards, leave the rows, or a chunk past max_chunk
    for cu in ([0, 2, 1, 9], [0, 2, 5, 12], [-1, 2, 5, 9], [0, 0, 5, 9]):
        out, err = run(cu=torch.tensor(cu, dtype=torch.int32))
        assert err & B.DEVERR_CHUNK, cu
        assert torch.equal(out[9:], c["out"][9:]) or cu[-1] > 9


@pytest.mark.parametrize("layout", [
    (2, 2, 128, 16, BF16, "io"), (2, 1, 64, 16, F16, "io"), (2, 1, 128, 4, F16, "io"),
    (2, 2, 128, 16, F16, "e4m3"),
], ids=str)
@pytest.mark.parametrize("chunks,tiles", [([5, 60], 1), ([200, 40], 1), ([200, 40], 2), ([200, 40], 3)],
                         ids=str)
def test_waits_that_run_out_are_reported_and_recoverable(layout, chunks, tiles):
    """Scores of a row tile withheld (the test hook): its softmax warps' waits run out, the other
    tile's warps give up wherever they are (some of them in their turns), nothing is written,
    the error word says so and the next call is right."""
    hq, hkv, d, bs, dtype, kind = layout
    c = chunk_case(2, hq, hkv, d, bs, dtype, chunks, [700, 130], kind, seed=5)
    g = on_gpu(c)
    part = 1024                                        # one partition: nothing is merged
    before = g["out"].clone()
    B.pa_testing_withhold_chunk_scores(tiles)
    try:
        out = call(g, partition_tokens=part)
        torch.cuda.synchronize()
        assert B.pa_get_device_error() == B.DEVERR_TIMEOUT
    finally:
        B.pa_testing_withhold_chunk_scores(0)
    # (a CTA whose only tile is not withheld is done as ever)
    rows = slice(0, 128 // (hq // hkv)) if tiles & 1 else slice(0, 0)
    assert torch.equal(out[rows][:chunks[0]], before[rows][:chunks[0]])
    got = call(g, partition_tokens=part)
    torch.cuda.synchronize()
    assert B.pa_get_device_error() == 0
    check(c, got)


def test_waits_that_run_out_in_a_split_context():
    c = chunk_case(1, 4, 2, 64, 16, F16, [3], [900], seed=6)
    g = on_gpu(c)
    B.pa_testing_withhold_chunk_scores(1)
    try:
        call(g, partition_tokens=128)
        torch.cuda.synchronize()
        assert B.pa_get_device_error() == B.DEVERR_TIMEOUT
    finally:
        B.pa_testing_withhold_chunk_scores(0)
    got = call(g, partition_tokens=128)
    torch.cuda.synchronize()
    assert B.pa_get_device_error() == 0
    check(c, got)


@pytest.mark.parametrize("kind,d,partition_tokens", [
    ("io", 64, 0), ("io", 128, 512), ("e4m3", 64, 0), ("e4m3", 128, 512)])
@pytest.mark.parametrize("down", [18.0, 22.0, 26.0])
def test_a_long_history_behind_one_large_score(kind, d, partition_tokens, down):
    """One token's score is `down` bits above all others and its V is zero: the row is the sum of
    2000 small weights. With P in f16 relative to a reference 7 to 15 bits below the maximum, a
    weight of w (of the largest) is off by at most 2^-11 w or half of f16's smallest step,
    2^-25 2^-7 = 2^-32: that much of each |v| more than the bound of chunk_plain."""
    n = 2000
    c = chunk_case(1, 2, 1, d, 16, F16, [2], [n], kind, seed=8, junk=False)
    c["q"].zero_()
    c["q"][:, :, 0] = 1.0
    sink = 700
    at = (int(c["tables"][0, sink // 16]), sink % 16)
    size = down * math.log(2) / c["scale"]              # q.K of the sink, the others' is 0
    if kind == "e4m3":
        c["k"].zero_()
        c["k_scale"].fill_(size / 448)
        c["k"][at[0], at[1], 0, 0] = 0x7e                # 448
        c["v"][:] = 0x78                                 # 256
        c["v_scale"].fill_(0.25)
    else:
        c["k"].zero_()
        c["k"][at[0], at[1], 0, 0] = size
        c["v"].fill_(64.0)
    c["v"][at[0], at[1]] = 0
    got = call(on_gpu(c), partition_tokens=partition_tokens)
    torch.cuda.synchronize()
    assert B.pa_get_device_error() == 0
    want, bound = attend_chunk(c["q"], c["k"], c["v"], c["cu"], c["tables"], c["lens"], c["scale"],
                               c["out"], 0, c["k_scale"], c["v_scale"])
    assert float(want.abs().min()) > 64 * n * 2.0 ** -(down + 1)
    bound = bound + n * 64 * 2.0 ** -32
    assert float(bound.max()) < 0.1 * float(want.abs().min())      # (the bound says something)
    assert bool(((got.cpu().double() - want).abs() <= bound).all())


@pytest.mark.parametrize("kind", ["io", "e4m3"])
def test_rows_before_the_first_sequence_stay(kind):
    """cu_chunk may start behind row 0: the rows in front are left as they were."""
    for chunks, lead in (([3, 0, 5], 7), ([140, 2, 1], 300)):
        c = chunk_case(3, 4, 2, 64, 16, F16, chunks, [200, 9, 150], kind, seed=12)
        rows = c["q"].shape[0]
        g2 = torch.Generator().manual_seed(1)
        for name in ("q", "out"):
            c[name] = torch.cat([torch.randn((lead, 4, 64), generator=g2).to(F16), c[name]])
        c["cu"] = c["cu"] + lead
        got = call(on_gpu(c))
        torch.cuda.synchronize()
        assert B.pa_get_device_error() == 0 and got.shape[0] == rows + lead
        check(c, got)
        assert torch.equal(got[:lead].cpu(), c["out"][:lead])


def test_no_rows_at_all():
    c = chunk_case(2, 4, 2, 64, 16, F16, [0, 0], [5, 0], pad=3)
    c["max_chunk"] = 0
    got = call(on_gpu(c))
    assert torch.equal(got.cpu(), c["out"])
    empty = dict(c, q=c["q"][:0], out=c["out"][:0])
    assert call(on_gpu(empty)).shape[0] == 0
    c["max_chunk"] = 4                                    # (an upper bound)
    assert torch.equal(call(on_gpu(c)).cpu(), c["out"]) and B.pa_get_device_error() == 0


@pytest.mark.parametrize("layout,bad", [
    ((2, 2, 128, 16, BF16, "io"), "nan"), ((2, 2, 128, 16, BF16, "io"), "inf"),
    ((4, 2, 64, 16, F16, "io"), "nan"), ((4, 2, 64, 16, F16, "io"), "-inf"),
    ((3, 1, 128, 4, F16, "io"), "nan"), ((3, 1, 128, 4, F16, "io"), "inf"),
    ((2, 1, 128, 16, F16, "e4m3"), "nan"), ((4, 4, 64, 32, BF16, "e4m3"), "nan")], ids=str)
@pytest.mark.parametrize("chunks,ctxs,window,part", [
    ([5, 9], [200, 70], 0, 0), ([300, 40], [420, 40], 0, 0), ([5, 9], [900, 300], 0, 128),
    ([150, 4], [400, 90], 50, 0), ([7], [700], 100, 128)], ids=str)
def test_values_of_tokens_a_row_does_not_see(layout, chunks, ctxs, window, part, bad):
    """V of new tokens that is not finite reaches only the rows that see it, and there only its
    own channels (so it is for tokens that the window of later rows drops)."""
    hq, hkv, d, bs, dtype, kind = layout
    c = chunk_case(len(chunks), hq, hkv, d, bs, dtype, chunks, ctxs, kind, seed=13)
    clean = c["v"].clone()
    v = c["v"].clone()
    # tokens of sequence 0 (positions) and the channels where V is bad
    n, L = chunks[0], ctxs[0]
    first = L - n                                      # the first new token's position
    spots = {L - 1: [0, d - 1], L - 1 - n // 3: [5], first + 1: [33, 34], first: [33]}
    if window:
        spots[max(0, first - window + 1)] = [7]        # seen by the first row alone
    for pos, channels in spots.items():
        at = int(c["tables"][0, pos // bs]), pos % bs
        for ch in channels:
            v[at[0], at[1], :, ch] = 0x7f if kind == "e4m3" else float(bad)
    g = on_gpu(dict(c, v=v))
    got = call(g, window=window, partition_tokens=part)
    place = call(g, window=window, partition_tokens=part, out=g["q"])      # in place
    torch.cuda.synchronize()
    assert B.pa_get_device_error() == 0
    assert torch.equal(got.nan_to_num(), place.nan_to_num())
    got = got.cpu().double()
    # what a row sees of the bad spots; zeros in their places for those that see none
    zero = v.clone()
    zero[~torch.isfinite(v.view(torch.float8_e4m3fn).double() if kind == "e4m3" else v.double())] = 0
    for name in ("clean", "zero"):
        want, bound = attend_chunk(c["q"], c["k"], clean if name == "clean" else zero, c["cu"],
                                   c["tables"], c["lens"], c["scale"], c["out"], window,
                                   c["k_scale"], c["v_scale"])
        for b in range(len(chunks)):
            for i in range(chunks[b]):
                r, pos = int(c["cu"][b]) + i, ctxs[b] - chunks[b] + i
                lo = max(0, pos - window + 1) if window else 0
                sees = torch.zeros(d, dtype=torch.bool)
                if b == 0:
                    for p, channels in spots.items():
                        if lo <= p <= pos:
                            sees[channels] = True
                assert not bool(torch.isfinite(got[r][:, sees]).any()), (b, i)
                err = (got[r] - want[r]).abs()[:, ~sees]
                assert bool((err <= bound[r][:, ~sees]).all()), (name, b, i)
