"""Prompts that PagedKVCache.add_sequence placed, attended with plan_chunk on
the GPU: prefixes served from the prefix cache, prompts in pieces, a prompt
that is cached whole, with a window. Outputs are held to float64 attention
over the logical history (the bound of tests/chunk_plain.py)."""
import pytest
import torch

from chunk_plain import attend_chunk
from paged_kv_cache_410_b200 import binding as B
from test_gpu_speculative import BS, D, HKV, HQ, Server

pytestmark = pytest.mark.gpu


def attend(s, plan, kv):
    """Run a plan whose tokens' K/V rows `kv` lists, and hold the result to float64. s.kv[id] is the
    sequence's whole history, a row (k, v) per token."""
    t = int(plan.counts.sum())
    q = s.rand(t, HQ, D)
    k, v = (torch.stack([r[i] for r in kv]) for i in (0, 1))
    dev = [x.cuda() for x in (q, k, v)]
    torch.cuda.synchronize()
    out = s.cache.attend_chunk(plan, 0, *dev)
    torch.cuda.synchronize()
    assert B.pa_get_device_error() == 0
    lens = plan.lengths.tolist()
    pools = []
    for which in (0, 1):
        pool = torch.zeros((len(lens), max(lens), HKV, D), dtype=torch.float64)
        for i, (sid, n) in enumerate(zip(plan.seq_ids.tolist(), lens)):
            rows = torch.stack([r[which] for r in s.kv[sid][:n]])
            pool[i, :n] = s.stored(rows, which)
        pools.append(pool)
    want, bound = attend_chunk(q, pools[0], pools[1], plan.cu_chunk.cpu(), [[i] for i in range(len(lens))],
                               lens, D ** -0.5, torch.zeros_like(q), s.window)
    if s.e4m3:   # q * k_scale in f16: as in tests/test_gpu_speculative.py
        size = float(q.double().abs().amax() * pools[0].abs().amax()) * D * D ** -0.5
        bound = bound + 2 * size * 2.0 ** -11 * float(pools[1].abs().amax())
    err = (out.cpu().double() - want).abs()
    assert bool((err <= bound).all()), float((err - bound).max())


@pytest.mark.parametrize("mode", ["f16", "bf16", "e4m3"])
def test_prompts_with_cached_prefixes(mode):
    s = Server(torch.bfloat16 if mode == "bf16" else torch.float16, mode == "e4m3", 0, seed=21)
    if mode == "e4m3":
        s.calibrate()

    def rows(n):
        return list(zip(s.rand(n, HKV, D), s.rand(n, HKV, D)))

    shared = list(range(70))
    assert s.cache.add_sequence(0, shared + [200, 201, 202])[0] == 0
    s.kv[0] = rows(73)
    # in two pieces
    attend(s, s.cache.plan_chunk([0], [0], [40]), s.kv[0][:40])
    attend(s, s.cache.plan_chunk([0], [40]), s.kv[0][40:])
    # two prompts with the same beginning: four whole blocks of it are there
    for sid, n in ((1, 150), (2, 1)):
        cached, _ = s.cache.add_sequence(sid, shared + list(range(300 + 200 * sid, 300 + 200 * sid + n)))
        assert cached == 64
        s.kv[sid] = s.kv[0][:64] + rows(6 + n)
        attend(s, s.cache.plan_chunk([sid], [64]), s.kv[sid][64:])
    # a prompt that is cached whole: its last row alone, nothing is stored again
    cached, slots = s.cache.add_sequence(3, shared[:64])
    assert cached == 64 and len(slots) == 0
    s.kv[3] = s.kv[0][:64]
    before = s.cache.k[0].clone(), s.cache.v[0].clone()
    attend(s, s.cache.plan_chunk([3, 1], [63, 180], [1, 2], stored=[64, 182]),
           rows(3))                                # (the K/V given for stored tokens is not read)
    assert torch.equal(before[0].view(torch.uint8), s.cache.k[0].view(torch.uint8))
    assert torch.equal(before[1].view(torch.uint8), s.cache.v[0].view(torch.uint8))
    # and the sequences go on
    s.speculate([0, 1, 2, 3])
    s.chunk([3, 0], [list(range(20)), [5]])
    for sid in range(4):
        s.read_back(sid)


def test_a_windowed_prompt_in_pieces():
    s = Server(torch.float16, False, 40, seed=22)
    s.cache.add_sequence(0, list(range(200)))
    s.kv[0] = list(zip(s.rand(200, HKV, D), s.rand(200, HKV, D)))
    free = s.cache.bm.num_free_blocks
    for first in range(0, 200, 50):
        attend(s, s.cache.plan_chunk([0], [first], [50]), s.kv[0][first:first + 50])
    assert s.cache.bm.num_free_blocks + s.cache.bm.num_cached_blocks >= free + (150 - 40) // BS
    s.chunk([0], [[1, 2, 3]])
    s.read_back(0)
