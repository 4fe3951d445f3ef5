"""Chunk attention and read-back at sizes the other tests stay below: contexts of
thousands of tokens (many laps of the kernel's ring, whole and split), caches
whose offsets pass 32 bits, read-backs of many CTAs of 32 rows, and the
two-launch batch captured into a graph. Against float64 row by row
(tests/chunk_plain.py), or bit for bit against the same tokens in a small cache."""
import pytest
import torch

from chunk_plain import U, chunk_case, on_gpu, paged_rows
from paged_kv_cache_410_b200 import binding as B
from test_gpu_chunk import BF16, F16, cache_of, call, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", [
    (4, 2, 128, 16, BF16, "io"), (3, 1, 64, 32, F16, "io"), (2, 2, 128, 4, F16, "io"),
    (4, 2, 128, 16, F16, "e4m3"), (4, 2, 64, 16, BF16, "e4m3")], ids=str)
@pytest.mark.parametrize("chunks,ctxs,window,part", [
    ([150, 1, 33], [6000, 4100, 2500], 0, 0), ([5, 1], [9000, 3001], 0, 0),
    ([5, 1], [9000, 3001], 0, 1 << 14), ([150, 2], [5000, 3000], 1500, 0)], ids=str)
def test_long_contexts(layout, chunks, ctxs, window, part):
    hq, hkv, d, bs, dtype, kind = layout
    c = chunk_case(len(chunks), hq, hkv, d, bs, dtype, chunks, ctxs, kind, pad=1, seed=9)
    got = call(on_gpu(c), window=window, partition_tokens=part)
    torch.cuda.synchronize()
    assert B.pa_get_device_error() == 0
    check(c, got, window)
    assert torch.equal(got[-1:].cpu(), c["out"][-1:])


def far(g, kind, bs, hkv, d):
    """The same tokens at the end of a cache whose offsets (elements, bytes of E4M3) pass 2^32."""
    nb = g["k"].shape[0]
    size = (1 << 32) // (bs * hkv * d) + 50
    f = dict(g)
    for name in ("k", "v"):
        big = torch.empty((size, bs, hkv, d), dtype=g[name].dtype, device="cuda")
        big[:100].fill_(0x7f if kind == "e4m3" else float("nan"))
        big[size - nb:] = g[name]
        f[name] = big
    live = g["tables"] < nb
    f["tables"] = torch.where(live, g["tables"] + (size - nb), g["tables"])
    return f


@pytest.mark.parametrize("layout", [(8, 4, 128, 16, BF16, "io"), (4, 4, 128, 4, F16, "io"),
                                    (8, 4, 128, 16, F16, "e4m3")], ids=str)
def test_offsets_past_32_bits(layout):
    hq, hkv, d, bs, dtype, kind = layout
    for chunks, ctxs in (([3, 1], [700, 90]), ([200, 5], [300, 40])):
        g = on_gpu(chunk_case(2, hq, hkv, d, bs, dtype, chunks, ctxs, kind, seed=11))
        want = call(g)
        f = far(g, kind, bs, hkv, d)
        assert f["k"].numel() > 1 << 32
        assert torch.equal(call(f), want)
        i32 = dict(dtype=torch.int32, device="cuda")
        rows = []
        for x in (g, f):
            k = torch.zeros((sum(ctxs), hkv, d), dtype=dtype, device="cuda")
            v = torch.zeros_like(k)
            B.pa_gather_kv(x["k"], x["v"], x["tables"], torch.tensor([0, 0], **i32),
                           torch.tensor([0, ctxs[0], sum(ctxs)], **i32), k, v, cache_of(x))
            rows += [(k, v)]
        assert torch.equal(rows[0][0], rows[1][0]) and torch.equal(rows[0][1], rows[1][1])
        assert B.pa_get_device_error() == 0
        del f, g, want, rows
        torch.cuda.empty_cache()


@pytest.mark.parametrize("cache", ["io", "e4m3"])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("tokens", [9471, 9472, 10003])
def test_gather_of_many_rows(cache, dtype, tokens):
    """32 rows a CTA from 9472 tokens on, eight below; sequences that begin and end inside a CTA's
    rows, empty ones among them, padding behind them."""
    ctxs = [4000, 33, 0, 2500, 1, tokens - 6534 + 10]
    first = [0, 0, 0, 0, 0, 10]
    c = chunk_case(6, 2, 2, 64, 16, dtype, [1] * 6, ctxs, cache, seed=tokens)
    cu = [0]
    for n, f in zip(ctxs, first):
        cu.append(cu[-1] + n - f)
    assert cu[-1] == tokens
    g = on_gpu(c)
    old = torch.randn((tokens + 3, 2, 64)).to(dtype)
    k, v = old.cuda(), old.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    B.pa_gather_kv(g["k"], g["v"], g["tables"], torch.tensor(first, **i32), torch.tensor(cu, **i32),
                   k, v, cache_of(g))
    assert B.pa_get_device_error() == 0
    for name, got in (("k", k.cpu()), ("v", v.cpu())):
        for b, (n, f) in enumerate(zip(ctxs, first)):
            rows = paged_rows(c[name], c[name + "_scale"], c["tables"][b], 16, n)[f:]
            x = got[cu[b]:cu[b + 1]].double()
            if cache == "io":
                assert torch.equal(x, rows)
            else:   # a float32 product, rounded once: half a step of each
                assert bool(((x - rows).abs() <= rows.abs() * (U[dtype] + 2.0 ** -23) + 2.0 ** -25).all())
        assert torch.equal(got[tokens:], old[tokens:])


@pytest.mark.parametrize("cache", ["io", "e4m3"])
def test_mixed_batch_of_many_captured(cache):
    """The two launches of a large mixed batch in a graph, replayed with other queries, chunks and
    lengths, with work behind it on the stream; two graphs replayed side by side."""
    chunks = [140 if i in (3, 38) else 70 if i == 17 else 1 for i in range(40)]
    ctxs = [n + (i * 13) % 90 for i, n in enumerate(chunks)]
    made = []
    for seed in (1, 2):
        c = chunk_case(40, 16, 8, 64, 16, F16, chunks, ctxs, cache, pad=2, seed=seed)
        g = on_gpu(c)
        out, copy = g["out"].clone(), torch.empty_like(g["out"])
        call(g, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(g, out=out, stream=torch.cuda.current_stream())
            copy.copy_(out)
        made.append((c, g, out, copy, graph))
    # another split of the batch: sequence 3 brings one token, sequence 0 none, all see less
    n2 = [0 if i == 0 else 1 if i == 3 else n for i, n in enumerate(chunks)]
    ctx2 = [max(n, L - 7) for n, L in zip(n2, ctxs)]
    cu2 = [0]
    for n in n2:
        cu2.append(cu2[-1] + n)
    streams = [torch.cuda.Stream() for _ in made]
    for c, g, out, copy, graph in made:
        c["q"] = torch.randn(c["q"].shape, generator=torch.Generator().manual_seed(7)).to(F16)
        c["cu"] = torch.tensor(cu2, dtype=torch.int32)
        c["lens"] = torch.tensor(ctx2, dtype=torch.int32)
        for name in ("q", "cu", "lens"):
            g[name].copy_(c[name])
        out.copy_(c["out"])
    torch.cuda.synchronize()
    for _ in range(3):
        for (c, g, out, copy, graph), s in zip(made, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert B.pa_get_device_error() == 0
    for c, g, out, copy, graph in made:
        check(c, copy)
        assert torch.equal(out, copy)
        assert torch.equal(copy[cu2[-1]:].cpu(), c["out"][cu2[-1]:])
