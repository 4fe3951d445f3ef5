"""The operators together, as a server uses them (PagedKVCache on the GPU):
an E4M3 cache calibrated before it is written, prompts run in chunks beside
sequences that decode, forks, speculative steps whose refused drafts leave the
cache, and the cache read back. Every attention output is held to float64
attention over the logical history (the bound of tests/chunk_plain.py), every
verification to its definition."""
import random

import pytest
import torch

from chunk_plain import attend_chunk, calibrate, verify_draft
from paged_kv_cache_410_b200 import binding as B
from paged_kv_cache_410_b200.kv_cache import PagedKVCache

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, VOCAB, MB = 8, 2, 64, 16, 300, 64


class Server:
    def __init__(self, dtype, e4m3, window, seed, stream=None):
        self.g = torch.Generator().manual_seed(seed)
        self.rng = random.Random(seed)
        self.dtype, self.window = dtype, window
        kw = {}
        if e4m3:
            ones = [torch.ones((HKV, D))]
            kw = dict(io_dtype=dtype, k_scales=ones, v_scales=ones)
        self.cache = PagedKVCache(256, BS, HKV, D, dtype=torch.uint8 if e4m3 else dtype,
                                  max_blocks_per_seq=MB, window=window, stream=stream, **kw)
        self.e4m3 = e4m3
        self.kv = {}        # logical K/V of each sequence's tokens: [(k, v)]

    def rand(self, *shape):
        return torch.randn(shape, generator=self.g).to(self.dtype)

    def calibrate(self):
        k, v = self.rand(200, HKV, D) * 2, self.rand(200, HKV, D) * 2
        self.cache.calibrate(0, k.cuda(), v.cuda())
        c = self.cache.layers[0]
        zero = torch.zeros((HKV, D))
        for x, s, i in ((k, c.k_scale, c.k_inv_scale), (v, c.v_scale, c.v_inv_scale)):
            _, scale, inv = calibrate(x, None, zero)
            assert torch.equal(s.cpu(), scale) and torch.equal(i.cpu(), inv)

    def stored(self, x, which):
        """What the cache holds of rows x: their bits, or their E4M3 codes times the scales."""
        if not self.e4m3:
            return x.double()
        c = self.cache.layers[0]
        s = (c.k_scale if which == 0 else c.v_scale).cpu()
        inv = (c.k_inv_scale if which == 0 else c.v_inv_scale).cpu()
        return (x.float() * inv).clamp(-448, 448).to(torch.float8_e4m3fn).double() * s.double()

    def chunk(self, ids, lists, drafts=False):
        plan = self.cache.begin_chunk(ids, lists, drafts=drafts)
        t = int(plan.counts.sum())
        q, k, v = self.rand(t, HQ, D), self.rand(t, HKV, D), self.rand(t, HKV, D)
        dev = [x.cuda() for x in (q, k, v)]
        torch.cuda.synchronize()
        out = self.cache.attend_chunk(plan, 0, *dev)
        torch.cuda.synchronize()
        assert B.pa_get_device_error() == 0
        at = 0
        for sid, run in zip(ids, lists):
            self.kv[sid] = self.kv.get(sid, []) + [(k[at + i], v[at + i]) for i in range(len(run))]
            at += len(run)
        # the same rows over a pool that holds each history in order
        lens = [len(self.kv[s]) for s in ids]
        most = max(lens)
        pools = []
        for which in (0, 1):
            rows = [torch.stack([kv[which] for kv in self.kv[s]]) if self.kv[s] else
                    torch.zeros((0, HKV, D), dtype=self.dtype) for s in ids]
            pool = torch.zeros((len(ids), most, HKV, D), dtype=torch.float64)
            for i, r in enumerate(rows):
                pool[i, :len(r)] = self.stored(r, which)
            pools.append(pool)
        cu = plan.cu_chunk.cpu()
        want, bound = attend_chunk(q, pools[0], pools[1], cu, [[i] for i in range(len(ids))], lens,
                                   D ** -0.5, torch.zeros_like(q), self.window)
        if self.e4m3:
            # q * k_scale is rounded to f16 in the kernel: 2^-11 of a score's products, of which
            # |q| |k| D bounds the sum; weights move by twice that
            size = float(q.double().abs().amax() * pools[0].abs().amax()) * D * D ** -0.5
            bound = bound + 2 * size * 2.0 ** -11 * float(pools[1].abs().amax())
        err = (out.cpu().double() - want).abs()
        assert bool((err <= bound).all()), float((err - bound).max())
        return plan

    def speculate(self, ids):
        lists = [[self.rng.randrange(VOCAB) for _ in range(self.rng.randint(1, 6))] for _ in ids]
        plan = self.chunk(ids, lists, drafts=True)
        t, n = int(plan.counts.sum()), len(ids)
        logits = torch.randn((t, VOCAB), generator=self.g)
        rows = [r for i in range(n) for r in range(int(plan.cu_chunk[i]), int(plan.cu_chunk[i + 1]) - 1)]
        target = torch.softmax(logits, -1)
        draft = torch.softmax(logits[rows] + 0.5 * torch.randn((len(rows), VOCAB), generator=self.g), -1)
        ua, us = torch.rand(len(rows), generator=self.g) * 0.6, torch.rand(n, generator=self.g)
        dev = [x.cuda() for x in (target, draft, ua, us)]
        torch.cuda.synchronize()
        accepted, tokens = self.cache.verify(plan, *dev)
        torch.cuda.synchronize()
        want = verify_draft(plan.drafts.cpu(), plan.cu_drafts.cpu(), target, draft, ua, us,
                            tokens.shape[1] - 1)
        assert accepted.tolist() == want[0] and tokens.tolist() == want[1]
        self.cache.settle(plan, accepted)
        for s, run, a in zip(ids, lists, want[0]):
            del self.kv[s][len(self.kv[s]) - len(run) + 1 + a:]
            assert self.cache.bm.length(s) == len(self.kv[s])

    def read_back(self, sid):
        first = 0
        n = len(self.kv[sid])
        if self.window:
            first = max(0, n - self.window)
        k, v = self.cache.read(0, sid, first, n - first)
        torch.cuda.synchronize()
        for which, got in ((0, k), (1, v)):
            want = self.stored(torch.stack([kv[which] for kv in self.kv[sid][first:]]), which)
            if self.e4m3:
                want = want.float().to(self.dtype)
            assert torch.equal(got.cpu().double(), want.double())


@pytest.mark.parametrize("mode", ["f16", "bf16", "e4m3", "window", "stream"])
def test_serving(mode):
    dtype = torch.bfloat16 if mode == "bf16" else torch.float16
    stream = torch.cuda.Stream() if mode == "stream" else None
    s = Server(dtype, mode == "e4m3", 40 if mode == "window" else 0, seed=len(mode), stream=stream)
    if mode == "e4m3":
        s.calibrate()
    for sid in range(4):
        s.cache.add_sequence(sid, [])
    # prompts in chunks, of different lengths, one of them late
    s.chunk([0, 1, 2], [list(range(150)), [7], list(range(33))])
    s.chunk([2, 0, 3], [list(range(20)), [1], list(range(70))])
    s.speculate([0, 1, 2, 3])
    if not s.window:
        s.cache.fork(0, 9)
        s.kv[9] = list(s.kv[0])
        s.speculate([9, 0, 2])
    for _ in range(3):
        s.speculate(s.rng.sample(list(s.kv), 3))
    # a mixed batch: a prompt's chunk beside single tokens
    s.chunk([1, 0, 3], [list(range(90)), [4], [5]])
    for sid in s.kv:
        s.read_back(sid)


def test_decode_continues_after_refused_drafts():
    """A plain decode step after speculative ones sees exactly the tokens that were kept."""
    s = Server(torch.float16, False, 0, seed=77)
    for sid in (0, 1):
        s.cache.add_sequence(sid, [])
    s.chunk([0, 1], [list(range(31)), list(range(5))])
    s.speculate([0, 1])
    plan = s.cache.begin_step([0, 1], [3, 4])
    q, k, v = s.rand(2, HQ, D), s.rand(2, HKV, D), s.rand(2, HKV, D)
    out = s.cache.attend(plan, 0, q.cuda(), k.cuda(), v.cuda())
    torch.cuda.synchronize()
    for i in (0, 1):
        s.kv[i].append((k[i], v[i]))
        kk = torch.stack([x[0] for x in s.kv[i]]).double()
        vv = torch.stack([x[1] for x in s.kv[i]]).double()
        for h in range(HQ):
            w = torch.softmax(kk[:, h // 4] @ q[i, h].double() * D ** -0.5, 0)
            want = w @ vv[:, h // 4]
            # P and the result in f16, scores of 32-bit sums (as in tests/chunk_plain.py)
            bound = (w @ vv[:, h // 4].abs()) * (2 ** -11 + 2 ** -14) + want.abs() * 2 ** -11 + 2 ** -24
            assert bool(((out[i, h].cpu().double() - want).abs() <= bound).all())
