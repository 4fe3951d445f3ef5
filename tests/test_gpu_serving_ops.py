"""Verification of drafts, calibration of an E4M3 cache's scales and the
read-back of cached tokens on the GPU, against their definitions in 64 bits
on the CPU (tests/chunk_plain.py). Tokens, counts, maxima, scales and a
16-bit cache's rows have to be equal; a dequantised value is a float32
product rounded to 16 bits: half a step of each."""
import pytest
import torch

from chunk_plain import U, calibrate, chunk_case, on_gpu, paged_rows, verify_draft
from paged_kv_cache_410_b200 import binding as B

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def run_verify(drafts, cu, target, draft, ua, us, most, stream=None, guard=0):
    batch = len(cu) - 1
    accepted = torch.full((batch,), -7, dtype=torch.int32, device="cuda")
    tokens = torch.full((batch, most + 1), -7, dtype=torch.int32, device="cuda")
    B.pa_verify_draft(drafts.cuda(), torch.tensor(cu, dtype=torch.int32, device="cuda"),
                      target.cuda(), None if draft is None else draft.cuda(), ua.cuda(),
                      us.cuda(), accepted, tokens, stream=stream)
    return accepted.tolist(), tokens.tolist()


def draft_case(counts, vocab, dtype, spread, seed):
    g = torch.Generator().manual_seed(seed)
    n, b = sum(counts), len(counts)
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    logits = torch.randn((n + b, vocab), generator=g) * spread
    target = torch.softmax(logits, -1)
    rows = [cu[s] + s + i for s in range(b) for i in range(counts[s])]
    draft = torch.softmax(logits[rows] + 0.3 * spread * torch.randn((n, vocab), generator=g), -1)
    drafts = torch.multinomial(draft, 1, generator=g).reshape(n).int() if n else torch.zeros(0, dtype=torch.int32)
    return (drafts, cu, target.to(dtype), draft.to(dtype), torch.rand(n, generator=g),
            torch.rand(b, generator=g))


@pytest.mark.parametrize("vocab", [1, 2, 127, 1000, 4096, 32000, 50257])
@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("has_q", [True, False])
def test_verify(vocab, dtype, has_q):
    counts = [3, 0, 1, 5, 4, 40, 0, 2]
    drafts, cu, target, draft, ua, us = draft_case(counts, vocab, dtype, 2.0, vocab)
    if not has_q:
        draft = None
    got = run_verify(drafts, cu, target, draft, ua, us, 40)
    assert B.pa_get_device_error() == 0
    want = verify_draft(drafts, cu, target, draft, ua, us, 40)
    assert got[0] == want[0]
    assert got[1] == want[1]


@pytest.mark.parametrize("batch", [37, 38, 74, 75, 148, 149, 160])
@pytest.mark.parametrize("vocab", [1, 5, 64, 1003, 2048])
@pytest.mark.parametrize("has_q", [True, False])
def test_verify_every_cluster_size(batch, vocab, has_q):
    """A sequence is taken by a cluster of 8, 4, 2 or 1 CTAs, by the batch: both sides of each
    border, for vocabularies whose warps reach the exchange at once, and without drafts."""
    counts = [(0, 2, 1, 4, 0, 0, 3)[i % 7] for i in range(batch)]
    for dtype in (F32, BF16):
        drafts, cu, target, draft, ua, us = draft_case(counts, vocab, dtype, 2.0, batch + vocab)
        ua *= 0.7
        if not has_q:
            draft = None
        want = verify_draft(drafts, cu, target, draft, ua, us, 4)
        for _ in range(2):
            got = run_verify(drafts, cu, target, draft, ua, us, 4)
            assert B.pa_get_device_error() == 0
            assert got[0] == want[0]
            assert got[1] == want[1]


def test_verify_nothing_left_of_the_difference():
    """p <= q everywhere (rows need not be normalised): the draw is from p."""
    drafts, cu, target, draft, ua, us = draft_case([2, 2], 513, F32, 1.0, 3)
    draft = torch.cat([target[:2], target[3:5]]) * 2
    ua = torch.full((4,), 0.75)
    got = run_verify(drafts, cu, target, draft, ua, us, 2)
    assert got == verify_draft(drafts, cu, target, draft, ua, us, 2)
    assert got[0] == [0, 0] and B.pa_get_device_error() == 0


@pytest.mark.parametrize("u", [0.0, 0.125, 0.5, 0.875, 1 - 2 ** -24])
@pytest.mark.parametrize("vocab", [8, 1024])
def test_verify_borders(u, vocab):
    """Equal weights with zeros between them: a draw on a border takes the token behind it."""
    target = torch.zeros((1, vocab))
    target[0, ::2] = 1.0 / vocab
    us = torch.tensor([u])
    none = torch.zeros(0, dtype=torch.int32)
    got = run_verify(none, [0, 0], target, None, torch.zeros(0), us, 0)
    assert got[0] == [0]
    assert got[1] == [[2 * int(u * (vocab // 2))]]


def test_verify_low_parts_of_the_differences():
    """p - q = 1 - 2^-25 and 2^-25 - 2^-50 side by side, then apart: half of the total is reached
    exactly behind the first two, so the draw is the next token. The first two's low parts, -2^-25
    and -2^-50, need 26 bits together."""
    p, q = torch.zeros((2, 12)), torch.zeros((1, 12))
    for i, j in ((0, 1), (4, 8)):
        p[0, i], q[0, i] = 1.0, 2.0 ** -25
        p[0, j], q[0, j] = 2.0 ** -25, 2.0 ** -50
    x = torch.tensor([2], dtype=torch.int32)             # weightless: refused
    u = torch.tensor([0.5])
    want = verify_draft(x, [0, 1], p, q, u, u, 1)
    assert want == ([0], [[4, -1]])
    assert run_verify(x, [0, 1], p, q, u, u, 1) == want


def test_verify_accept_border_is_strict():
    """u q = p refuses, one step less accepts."""
    target = torch.tensor([[0.25, 0.75], [0.5, 0.5]])
    draft = torch.tensor([[0.5, 0.5]])
    x = torch.tensor([0], dtype=torch.int32)
    us = torch.tensor([0.1])
    for u, kept in ((0.5, 0), (0.5 - 2 ** -25, 1)):
        assert run_verify(x, [0, 1], target, draft, torch.tensor([u]), us, 1)[0] == [kept]


def test_verify_values_that_count_as_zero():
    drafts, cu, target, draft, ua, us = draft_case([4, 4, 4], 999, F32, 1.0, 9)
    for k, bad in enumerate((float("nan"), float("inf"), -1.0, float("-inf"))):
        target[k::7, 5 + k::11] = bad
        draft[k::5, 3 + k::13] = bad
    got = run_verify(drafts, cu, target, draft, ua, us, 4)
    assert got == verify_draft(drafts, cu, target, draft, ua, us, 4)
    assert B.pa_get_device_error() == 0


def test_verify_reports_bad_values():
    drafts, cu, target, draft, ua, us = draft_case([2, 3], 100, F32, 1.0, 4)
    ua.zero_()
    bad = drafts.clone()
    bad[1] = 100
    got = run_verify(bad, cu, target, draft, ua, us, 3)
    assert B.pa_get_device_error() == B.DEVERR_TOKEN
    assert got == verify_draft(bad, cu, target, draft, ua, us, 3) and got[0][0] == 1
    # a row without weight: token -1, the other sequence as it was
    t = target.clone()
    t[2] = 0.0
    got = run_verify(drafts, cu, t, draft, ua, us, 3)
    assert B.pa_get_device_error() == B.DEVERR_PROBS
    assert got[1][0] == drafts[:2].tolist() + [-1, -1]
    assert got == verify_draft(drafts, cu, t, draft, ua, us, 3)
    # row starts that run backwards, leave the rows, or a sequence past max_drafts: untouched
    for cu2, most in (([0, 3, 2], 3), ([0, 2, 6], 4), ([-1, 2, 5], 3), ([0, 2, 5], 2)):
        got = run_verify(drafts, cu2, target, draft, ua, us, most)
        assert B.pa_get_device_error() == B.DEVERR_CHUNK, cu2
        assert -7 in got[0]


def test_verify_captured_on_two_streams():
    """Two captured calls replayed side by side share nothing."""
    cases = [draft_case([3] * 20, 5000, F32, 2.0, s) for s in (1, 2)]
    graphs, outs, keep = [], [], []
    for c in cases:
        dev = [x.cuda() if isinstance(x, torch.Tensor) else torch.tensor(x, dtype=torch.int32, device="cuda")
               for x in c]
        acc = torch.zeros(20, dtype=torch.int32, device="cuda")
        tok = torch.zeros((20, 4), dtype=torch.int32, device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            B.pa_verify_draft(dev[0], dev[1], dev[2], dev[3], dev[4], dev[5], acc, tok,
                              stream=torch.cuda.current_stream())
        graphs.append(g)
        outs.append((acc, tok))
        keep.append(dev)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, (acc, tok) in zip(cases, outs):
        want = verify_draft(*c, 3)
        assert (acc.tolist(), tok.tolist()) == want


@pytest.mark.parametrize("tokens", [0, 1, 17, 300, 5000])
@pytest.mark.parametrize("heads", [(1, 64), (5, 128), (8, 128), (20, 128)], ids=str)
@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
def test_calibrate(tokens, heads, dtype):
    hkv, d = heads
    g = torch.Generator().manual_seed(tokens + hkv)
    big = 3e4 if dtype == F16 else 1e30
    arrays = {n: torch.rand((hkv, d), generator=g) for n in ("k_amax", "v_amax")}
    arrays["k_amax"][0, :5] = 0.0
    x = {}
    for n in "kv":
        t = torch.randn((tokens, hkv, d), generator=g).to(dtype)
        if tokens:
            t[0, 0, 0] = float("nan")
            t[tokens // 2, 0, 1] = float("inf")
            t[tokens // 2, 0, 2] = float("-inf")
            t[-1, 0, 3] = -big
            t[:, 0, 4] = 0.0
        x[n] = t
    slots = torch.arange(tokens)
    slots[torch.rand(tokens, generator=g) < 0.3] = -1
    for use in (slots, None):
        dev = {n: a.cuda() for n, a in arrays.items()}
        out = {f"{n}_{w}": torch.full((hkv, d), 9.0, device="cuda") for n in "kv" for w in ("scale", "inv_scale")}
        B.pa_calibrate_kv(x["k"].cuda(), x["v"].cuda(), None if use is None else use.cuda(),
                          dev["k_amax"], dev["v_amax"], out["k_scale"], out["v_scale"],
                          out["k_inv_scale"], out["v_inv_scale"])
        for n in "kv":
            amax, scale, inv = calibrate(x[n], use, arrays[n + "_amax"])
            assert torch.equal(dev[n + "_amax"].cpu(), amax)
            assert torch.equal(out[n + "_scale"].cpu(), scale)
            assert torch.equal(out[n + "_inv_scale"].cpu(), inv)


def test_calibrate_in_pieces_is_calibrate_at_once():
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn((700, 2, 64), generator=g).to(BF16).cuda() for _ in range(2))
    results = []
    for cuts in ([700], [1, 299, 400]):
        a = [torch.zeros((2, 64), device="cuda") for _ in range(6)]
        at = 0
        for n in cuts:
            B.pa_calibrate_kv(k[at:at + n], v[at:at + n], None, *a)
            at += n
        results.append(a)
    assert all(torch.equal(x, y) for x, y in zip(*results))


def test_calibrate_tiny_values_keep_finite_inverses():
    x = torch.full((4, 1, 64), 1e-38, dtype=BF16, device="cuda")
    a = [torch.zeros((1, 64), device="cuda") for _ in range(6)]
    B.pa_calibrate_kv(x, x, None, *a)
    assert bool(torch.isfinite(a[4]).all()) and bool((a[2] == 2.0 ** -126).all())


@pytest.mark.parametrize("layout", [(1, 64, 16), (5, 128, 1), (8, 128, 256), (32, 128, 32), (2, 64, 4)], ids=str)
@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("cache", ["io", "e4m3"])
def test_gather(layout, dtype, cache):
    hkv, d, bs = layout
    ctxs = [1, 70, 0, 300, 33]
    first = [0, 13, 0, 255, 0]
    count = [1, 57, 0, 45, 0]
    c = chunk_case(5, hkv, hkv, d, bs, dtype, [1] * 5, ctxs, cache)
    cu = [0]
    for n in count:
        cu.append(cu[-1] + n)
    g = on_gpu(c)
    sc = {} if cache == "io" else dict(k_scale=g["k_scale"], v_scale=g["v_scale"],
                                       k_inv_scale=1 / g["k_scale"], v_inv_scale=1 / g["v_scale"])
    old = torch.randn((cu[-1] + 2, hkv, d), dtype=torch.float32).to(dtype)
    k, v = old.cuda(), old.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    B.pa_gather_kv(g["k"], g["v"], g["tables"], torch.tensor(first, **i32), torch.tensor(cu, **i32),
                   k, v, B.PagedCache.for_tensor(g["k"], **sc))
    assert B.pa_get_device_error() == 0
    for name, got in (("k", k.cpu()), ("v", v.cpu())):
        for b in range(5):
            rows = paged_rows(c[name], c[name + "_scale"], c["tables"][b], bs, first[b] + count[b])[first[b]:]
            x = got[cu[b]:cu[b + 1]]
            if cache == "io":
                assert torch.equal(x.double(), rows)
            else:
                err = (x.double() - rows).abs()
                assert bool((err <= rows.abs() * (U[dtype] + 2.0 ** -23) + 2.0 ** -25).all())
        assert torch.equal(got[cu[-1]:], old[cu[-1]:])


def test_gather_reports_bad_values():
    c = chunk_case(2, 2, 2, 64, 16, F16, [1, 1], [40, 50])
    g = on_gpu(c)
    cache = B.PagedCache.for_tensor(g["k"])
    i32 = dict(dtype=torch.int32, device="cuda")

    def run(first=(0, 0), cu=(0, 20, 40), tables=None):
        k = torch.full((40, 2, 64), 7.0, dtype=F16, device="cuda")
        v = k.clone()
        B.pa_gather_kv(g["k"], g["v"], g["tables"] if tables is None else tables,
                       torch.tensor(first, **i32), torch.tensor(cu, **i32), k, v, cache)
        return k.cpu(), B.pa_get_device_error()

    ok, err = run()
    assert err == 0
    k, err = run(first=(-5, 0))
    assert err == B.DEVERR_CONTEXT_LEN and bool((k[:5] == 0).all()) and torch.equal(k[20:], ok[20:])
    k, err = run(first=(0, 1000))
    assert err == B.DEVERR_CONTEXT_LEN and bool((k[20:] == 0).all()) and torch.equal(k[:20], ok[:20])
    t = g["tables"].clone()
    t[0, 1] = -1
    k, err = run(tables=t)
    assert err == B.DEVERR_BLOCK_ID and bool((k[16:20] == 0).all()) and torch.equal(k[:16], ok[:16])
    for cu in ((0, 30, 20), (0, 20, 41), (-1, 20, 40)):
        assert run(cu=cu)[1] & B.DEVERR_CHUNK


def test_round_trip_between_caches():
    """Rows read from one cache and appended to another of a different block size are the same
    tokens there."""
    c = chunk_case(1, 4, 4, 128, 16, BF16, [1], [100])
    g = on_gpu(c)
    k = torch.empty((100, 4, 128), dtype=BF16, device="cuda")
    v = torch.empty_like(k)
    i32 = dict(dtype=torch.int32, device="cuda")
    zero, cu = torch.tensor([0], **i32), torch.tensor([0, 100], **i32)
    B.pa_gather_kv(g["k"], g["v"], g["tables"], zero, cu, k, v, B.PagedCache.for_tensor(g["k"]))
    k2 = torch.zeros((9, 64, 4, 128), dtype=BF16, device="cuda")
    v2 = torch.zeros_like(k2)
    table = torch.tensor([[7, 2]], **i32)
    slots = torch.cat([torch.arange(64) + 7 * 64, torch.arange(36) + 2 * 64]).cuda()
    other = B.PagedCache.for_tensor(k2)
    B.pa_append_kv(k, v, slots, k2, v2, other)
    k3, v3 = torch.empty_like(k), torch.empty_like(v)
    B.pa_gather_kv(k2, v2, table, zero, cu, k3, v3, other)
    assert torch.equal(k, k3) and torch.equal(v, v3) and B.pa_get_device_error() == 0
