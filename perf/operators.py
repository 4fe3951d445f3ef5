"""The serving operators measured on a GPU: chunk attention over the paged cache, verification of
drafted tokens, calibration of an E4M3 cache's scales, and reading cached tokens back.

Each case is one call. `run` computes it in elementary torch operations, or, with `own`, through
the library's binding. Lengths come from a case's own sizes, tensor values from the seed.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
SMALLEST_SCALE = 2.0 ** -126  # the smallest normal float32: its reciprocal is finite
IO = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases --------------------------------------------------------------------------------------
def _attend(name, batch, heads, d, bs, io, chunk, past, cache="io", window=0, singles=0.0, pad=0):
    c = {"op": "attend", "batch": batch, "hq": heads[0], "hkv": heads[1], "d": d, "bs": bs,
         "io": io, "cache": cache, "chunk_lo": chunk[0], "chunk_hi": chunk[1],
         "past_lo": past[0], "past_hi": past[1], "window": window, "singles": singles, "pad": pad}
    return dict(c, name=name) if name else c


def _verify(name, batch, drafts, vocab, probs, spread, has_q=True):
    c = {"op": "verify", "batch": batch, "drafts": drafts, "vocab": vocab, "probs": probs,
         "spread": spread, "has_q": has_q}
    return dict(c, name=name) if name else c


def _gather(name, batch, hkv, d, bs, io, cache, tokens, pad=0):
    c = {"op": "gather", "batch": batch, "hkv": hkv, "d": d, "bs": bs, "io": io, "cache": cache,
         "tok_lo": tokens[0], "tok_hi": tokens[1], "pad": pad}
    return dict(c, name=name) if name else c


def _calibrate(name, tokens, hkv, d, io, padding):
    c = {"op": "calibrate", "tokens": tokens, "hkv": hkv, "d": d, "io": io, "padding": padding}
    return dict(c, name=name) if name else c


def listed():
    return [
        # four drafts and the last token of a few short requests, one small layer: launch latency
        _attend("attend-drafts-tiny", 4, (8, 8), 64, 16, "f16", (1, 5), (1, 200)),
        # a speculative step of a full batch, 8 query heads per KV head: every cached token is read
        _attend("attend-drafts-gqa", 64, (64, 8), 128, 16, "bf16", (2, 8), (512, 4096)),
        # two prompts in chunks of up to 2048, every head with its own KV head; rows of padding
        _attend("attend-prompt-mha", 2, (32, 32), 128, 16, "f16", (1700, 2048), (0, 2048), pad=5),
        # the last chunk of a long prompt
        _attend("attend-prompt-long", 1, (64, 8), 128, 16, "bf16", (2048, 2048), (14336, 14336)),
        # an E4M3 cache, one step of a mixed batch: most requests decode one token, some a chunk
        _attend("attend-mixed-e4m3", 32, (32, 8), 128, 32, "f16", (64, 512), (16, 4096),
                cache="e4m3", singles=0.7),
        # sliding window: a chunk whose history reaches past the window
        _attend("attend-window", 2, (32, 8), 128, 16, "bf16", (1000, 1024), (5000, 8000),
                window=4096),
        # drafts of a few requests, a 32000-token vocabulary
        _verify("verify-small", 4, 4, 32000, "f32", 3.0),
        # a full batch, 7 drafts each, a large vocabulary
        _verify("verify-large", 256, 7, 131072, "f32", 3.0),
        # one request's tokens read from an E4M3 cache, to move it to another cache
        _gather("gather-e4m3", 1, 8, 128, 16, "bf16", "e4m3", (600, 600)),
        # a batch swapped out of a 16-bit cache
        _gather("gather-batch", 64, 32, 128, 16, "f16", "io", (512, 4096), pad=3),
        # the scales of an E4M3 cache from a short prompt
        _calibrate("calibrate-small", 200, 8, 128, "f16", 0.1),
        # and from a calibration set of many prompts
        _calibrate("calibrate-large", 262144, 8, 128, "bf16", 0.02),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "verify", "gather", "calibrate"])
    if op == "attend":
        hkv = rng.choice([1, 2, 4, 5, 8, 32])
        hq = hkv * (1 if hkv == 32 else rng.choice([1, 2, 3, 4, 7, 8]))
        d = rng.choice([64, 128])
        hi = _log(rng, 1, 2048)
        lo = _log(rng, 1, hi)
        past = _log(rng, 1, 14336)
        batch = _log(rng, 1, 64)
        # the plain form's padded scores stay below the largest listed case's
        while batch > 1 and batch * hq * hi * (past + hi) > 2 ** 30:
            batch -= 1
        while batch * hq * hi * (past + hi) > 2 ** 31:
            past //= 2
            hi = max(lo, hi - hi // 4)
            lo = min(lo, max(1, hi // 2))
        window = rng.choice([0, 0, _log(rng, 1, 4096)])
        return _attend(None, batch, (hq, hkv), d, rng.choice([1, 4, 8, 16, 32, 64, 128, 256]),
                       rng.choice(["f16", "bf16"]), (lo, hi), (rng.choice([0, past // 2]), past),
                       cache=rng.choice(["io", "io", "e4m3"]), window=window,
                       singles=rng.choice([0.0, 0.0, 0.5]), pad=rng.choice([0, 0, 1, 6]))
    if op == "verify":
        vocab = _log(rng, 1000, 131072)
        batch = _log(rng, 1, 200)
        return _verify(None, batch, rng.randint(1, 8), vocab, rng.choice(["f32", "f32", "bf16", "f16"]),
                       rng.choice([1.0, 3.0, 6.0]), rng.choice([True, True, False]))
    if op == "gather":
        hi = _log(rng, 1, 4096)
        return _gather(None, _log(rng, 1, 48), rng.choice([1, 2, 5, 8, 32]), rng.choice([64, 128]),
                       rng.choice([1, 4, 16, 32, 128, 256]), rng.choice(["f16", "bf16"]),
                       rng.choice(["io", "e4m3"]), (_log(rng, 1, hi), hi), rng.choice([0, 1, 4]))
    return _calibrate(None, _log(rng, 1, 200000), rng.choice([1, 2, 5, 8]), rng.choice([64, 128]),
                      rng.choice(["f16", "bf16"]), rng.choice([0.0, 0.3]))


def _rng(case):
    """Lengths belong to the case, not to the seed."""
    return random.Random(str(sorted((k, v) for k, v in case.items() if k != "name")))


def _attend_lengths(case):
    """(new tokens, context with them) of each sequence."""
    r = _rng(case)
    new, ctx = [], []
    for _ in range(case["batch"]):
        n = 1 if r.random() < case["singles"] else r.randint(case["chunk_lo"], case["chunk_hi"])
        new.append(n)
        ctx.append(n + r.randint(case["past_lo"], case["past_hi"]))
    return new, ctx


def _draft_counts(case):
    r = _rng(case)
    return [r.randint(max(1, case["drafts"] - 2), case["drafts"]) for _ in range(case["batch"])]


def _gather_ranges(case):
    """(first position, tokens) of each sequence."""
    r = _rng(case)
    return ([r.randint(0, 40) for _ in range(case["batch"])],
            [r.randint(case["tok_lo"], case["tok_hi"]) for _ in range(case["batch"])])


def _starts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


# ---- inputs -------------------------------------------------------------------------------------
def _paged(case, lens, gen, dev):
    """Block tables over a shuffled pool, and K/V pools (with the scales of an E4M3 cache)."""
    bs, hkv, d = case["bs"], case["hkv"], case["d"]
    need = [-(-n // bs) for n in lens]
    total = max(1, sum(need))
    blocks = total + total // 10 + 1
    perm = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)
    tables = torch.zeros((len(lens), max(1, max(need))), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = perm[at:at + n]
        at += n
    shape = (blocks, bs, hkv, d)
    s = {"tables": tables, "scales": None}
    if case["cache"] == "e4m3":
        scales = []
        for name in ("k_cache", "v_cache"):
            # N(0, 1) codes times 90: the largest of many reach 448; channels differ in size
            x = torch.empty(shape, dtype=torch.float16, device=dev).normal_(generator=gen).mul_(90.0)
            s[name] = x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
            scales.append(torch.empty((hkv, d), device=dev).uniform_(0.5, 2.0, generator=gen) / 90.0)
        s["scales"] = [scales[0], scales[1], 1.0 / scales[0], 1.0 / scales[1]]
    else:
        for name in ("k_cache", "v_cache"):
            s[name] = torch.empty(shape, dtype=IO[case["io"]], device=dev).normal_(generator=gen)
    return s


def _i32(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 410)
    s = {"case": case}
    if case["op"] == "attend":
        new, ctx = _attend_lengths(case)
        s.update(_paged(case, ctx, gen, dev))
        rows = sum(new) + case["pad"]
        shape = (rows, case["hq"], case["d"])
        s["q"] = torch.empty(shape, dtype=IO[case["io"]], device=dev).normal_(generator=gen)
        s["out"] = torch.empty(shape, dtype=IO[case["io"]], device=dev).normal_(generator=gen)
        s["cu"], s["lens"] = _i32(_starts(new), dev), _i32(ctx, dev)
        s["max_new"], s["max_ctx"] = max(new), max(ctx)
        s["scale"] = 1.0 / math.sqrt(case["d"])
    elif case["op"] == "verify":
        counts = _draft_counts(case)
        n, b, v = sum(counts), case["batch"], case["vocab"]
        s["cu"] = _i32(_starts(counts), dev)
        target = torch.empty((n + b, v), device=dev).normal_(generator=gen).mul_(case["spread"])
        seq = torch.repeat_interleave(torch.arange(b, device=dev), torch.tensor(counts, device=dev), output_size=n)
        rows = torch.arange(n, device=dev) + seq  # the target row of each draft
        draft = target[rows] + torch.empty((n, v), device=dev).normal_(generator=gen).mul_(0.3 * case["spread"])
        draft = torch.softmax(draft, -1)
        drawn = torch.empty((n, 1), dtype=torch.float64, device=dev).uniform_(generator=gen)
        at = torch.searchsorted(torch.cumsum(draft.double(), -1), drawn, right=True).clamp_(max=v - 1)
        s["drafts"] = at.reshape(n).to(torch.int32)
        s["target_probs"] = torch.softmax(target, -1).to(IO[case["probs"]])
        s["draft_probs"] = draft.to(IO[case["probs"]]) if case["has_q"] else None
        s["u_accept"] = torch.empty(n, device=dev).uniform_(generator=gen)
        s["u_sample"] = torch.empty(b, device=dev).uniform_(generator=gen)
        s["accepted"] = torch.zeros(b, dtype=torch.int32, device=dev)
        s["tokens"] = torch.zeros((b, case["drafts"] + 1), dtype=torch.int32, device=dev)
    elif case["op"] == "gather":
        first, count = _gather_ranges(case)
        s.update(_paged(case, [f + c for f, c in zip(first, count)], gen, dev))
        s["first"], s["cu"] = _i32(first, dev), _i32(_starts(count), dev)
        shape = (sum(count) + case["pad"], case["hkv"], case["d"])
        for name in ("k_out", "v_out"):
            s[name] = torch.empty(shape, dtype=IO[case["io"]], device=dev).normal_(generator=gen)
    else:
        t, hkv, d = case["tokens"], case["hkv"], case["d"]
        size = torch.empty((1, hkv, d), device=dev).uniform_(0.25, 4.0, generator=gen)
        for name in ("k", "v"):
            x = torch.empty((t, hkv, d), dtype=IO[case["io"]], device=dev).normal_(generator=gen)
            s[name] = x.mul_(size.to(x.dtype))
        s["slots"] = torch.arange(t, device=dev)
        skip = torch.empty(t, device=dev).uniform_(generator=gen) < case["padding"]
        s["slots"].masked_fill_(skip, -1)
        # what earlier prompts have left
        for name in ("k_amax", "v_amax"):
            s[name] = torch.empty((hkv, d), device=dev).uniform_(0.0, 6.0, generator=gen)
        for name in ("k_scale", "v_scale", "k_inv_scale", "v_inv_scale"):
            s[name] = torch.zeros((hkv, d), device=dev)
    return s


# ---- plain forms --------------------------------------------------------------------------------
def _read(pool, scale, slots):
    """Cached rows at `slots` in float32."""
    rows = pool.reshape(-1, *pool.shape[2:])[slots]
    if scale is None:
        return rows.float()
    return rows.view(torch.float8_e4m3fn).float() * scale


def _attend_plain(s):
    c = s["case"]
    cu, lens = s["cu"].long(), s["lens"].long()
    dev, batch, n, L = cu.device, c["batch"], s["max_new"], s["max_ctx"]
    hkv, group, d = c["hkv"], c["hq"] // c["hkv"], c["d"]
    new = cu[1:] - cu[:-1]
    j = torch.arange(L, device=dev)
    valid = j[None, :] < lens[:, None]
    slots = torch.where(valid, s["tables"].long()[:, j // c["bs"]] * c["bs"] + j % c["bs"], 0)
    ks, vs = (None, None) if s["scales"] is None else s["scales"][:2]
    k = _read(s["k_cache"], ks, slots).permute(0, 2, 3, 1)                      # [B, Hkv, D, L]
    v = _read(s["v_cache"], vs, slots)
    v = torch.where(valid[:, :, None, None], v, 0.0).permute(0, 2, 1, 3)        # [B, Hkv, L, D]
    i = torch.arange(n, device=dev)
    row = (cu[:-1, None] + i[None, :]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float() * s["scale"]                                        # [B, n, Hq, D]
    q = q.reshape(batch, n, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, group * n, d)
    score = torch.matmul(q, k).reshape(batch, hkv, group, n, L)
    pos = lens[:, None] - new[:, None] + i[None, :]
    seen = (j[None, None, :] <= pos[:, :, None]) & valid[:, None, :]
    if c["window"]:
        seen = seen & (j[None, None, :] > pos[:, :, None] - c["window"])
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score.reshape(batch, hkv, group * n, L), v).reshape(batch, hkv, group, n, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(batch, n, c["hq"], d)
    t = torch.arange(s["out"].shape[0], device=dev)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=batch - 1)
    o = o[b, (t - cu[b]).clamp(max=n - 1)].to(s["out"].dtype)
    return torch.where((t < cu[-1])[:, None, None], o, s["out"])


def _verify_plain(s):
    c = s["case"]
    cu = s["cu"].long()
    dev, batch, most = cu.device, c["batch"], c["drafts"]
    n = cu[1:] - cu[:-1]
    i = torch.arange(most + 1, device=dev)
    b = torch.arange(batch, device=dev)
    total = s["drafts"].shape[0]
    has = i[None, :] < n[:, None]
    at = (cu[:-1, None] + i[None, :]).clamp(max=total - 1)
    token = s["drafts"].long()[at]
    p = s["target_probs"][(at + b[:, None]).clamp(max=total + batch - 1), token].double()
    q = s["draft_probs"][at, token].double() if c["has_q"] else 1.0
    passed = (s["u_accept"].double()[at] * q < p) & has
    accepted = torch.cumprod(passed.long(), -1).sum(-1)
    stop = (cu[:-1] + accepted).clamp(max=total - 1)
    full = accepted == n
    p = s["target_probs"][cu[:-1] + b + accepted].double()
    if c["has_q"]:
        q = s["draft_probs"][stop].double()
    else:
        q = torch.nn.functional.one_hot(s["drafts"].long()[stop], c["vocab"]).double()
    w = torch.where(full[:, None], p, (p - q).clamp(min=0.0))
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, p)
    cum = torch.cumsum(w, -1)
    pick = (cum <= s["u_sample"].double()[:, None] * cum[:, -1:]).sum(-1)
    v = torch.arange(c["vocab"], device=dev)
    last = torch.where(w > 0, v[None, :], -1).amax(-1)
    pick = torch.minimum(pick, last)
    out = torch.where(i[None, :] < accepted[:, None], token, -1)
    out = torch.where(i[None, :] == accepted[:, None], pick[:, None], out)
    return {"accepted": accepted.to(torch.int32), "tokens": out.to(torch.int32)}


def _gather_plain(s):
    c = s["case"]
    cu = s["cu"].long()
    t = torch.arange(s["k_out"].shape[0], device=cu.device)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=c["batch"] - 1)
    live = t < cu[-1]
    pos = torch.where(live, t - cu[b] + s["first"].long()[b], 0)
    slots = s["tables"].long()[b, pos // c["bs"]] * c["bs"] + pos % c["bs"]
    ks, vs = (None, None) if s["scales"] is None else s["scales"][:2]
    return {name: torch.where(live[:, None, None], _read(pool, sc, slots).to(old.dtype), old)
            for name, pool, sc, old in (("k", s["k_cache"], ks, s["k_out"]), ("v", s["v_cache"], vs, s["v_out"]))}


def _calibrate_plain(s):
    live = (s["slots"] >= 0)[:, None, None]
    out = {}
    for name in ("k", "v"):
        x = s[name].float().abs()
        x = torch.where(live & (x < math.inf), x, 0.0)
        amax = torch.maximum(s[name + "_amax"], x.amax(0))
        scale = torch.where(amax > 0, (amax / E4M3_MAX).clamp(min=SMALLEST_SCALE), 1.0)
        out.update({name + "_amax": amax, name + "_scale": scale, name + "_inv_scale": 1.0 / scale})
    return out


# ---- the library's calls ------------------------------------------------------------------------
def _cache(s, B):
    k, sc = s["k_cache"], s["scales"]
    if sc is None:
        return B.PagedCache.for_tensor(k)
    return B.PagedCache.for_tensor(k, k_scale=sc[0], v_scale=sc[1], k_inv_scale=sc[2], v_inv_scale=sc[3])


def _own(s):
    from paged_kv_cache_410_b200 import binding as B
    c = s["case"]
    if c["op"] == "attend":
        if "cache" not in s:
            s["cache"] = _cache(s, B)
            need = B.pa_attend_chunk_workspace_size(s["q"].shape[0], c["batch"], c["hq"], s["max_new"],
                                                    s["max_ctx"], s["cache"], window=c["window"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device=s["q"].device) if need else None
        B.pa_attend_chunk(s["q"], s["k_cache"], s["v_cache"], s["cu"], s["tables"], s["lens"], s["scale"],
                          s["out"], s["cache"], s["max_new"], s["max_ctx"], window=c["window"],
                          workspace=s["workspace"])
        return s["out"]
    if c["op"] == "verify":
        B.pa_verify_draft(s["drafts"], s["cu"], s["target_probs"], s["draft_probs"], s["u_accept"],
                          s["u_sample"], s["accepted"], s["tokens"])
        return {"accepted": s["accepted"], "tokens": s["tokens"]}
    if c["op"] == "gather":
        if "cache" not in s:
            s["cache"] = _cache(s, B)
        B.pa_gather_kv(s["k_cache"], s["v_cache"], s["tables"], s["first"], s["cu"], s["k_out"], s["v_out"],
                       s["cache"])
        return {"k": s["k_out"], "v": s["v_out"]}
    B.pa_calibrate_kv(s["k"], s["v"], s["slots"], s["k_amax"], s["v_amax"], s["k_scale"], s["v_scale"],
                      s["k_inv_scale"], s["v_inv_scale"])
    return {n: s[n] for n in ("k_amax", "k_scale", "k_inv_scale", "v_amax", "v_scale", "v_inv_scale")}


def run(state):
    if own:
        return _own(state)
    plain = {"attend": _attend_plain, "verify": _verify_plain, "gather": _gather_plain,
             "calibrate": _calibrate_plain}
    return plain[state["case"]["op"]](state)


# ---- what a pass needs --------------------------------------------------------------------------
def work(case):
    if case["op"] == "attend":
        new, ctx = _attend_lengths(case)
        w = case["window"] or max(ctx)
        elt = 1 if case["cache"] == "e4m3" else 2
        tokens = sum(min(L, n + w - 1) for n, L in zip(new, ctx))
        pairs = sum(sum(min(p, w) for p in range(L - n + 1, L + 1)) for n, L in zip(new, ctx))
        rows = sum(new) * case["hq"] * case["d"]
        table = sum(-(-min(L, n + w - 1) // case["bs"]) for n, L in zip(new, ctx))
        return {"bytes": 2 * 2 * rows + 2 * tokens * case["hkv"] * case["d"] * elt + 4 * table
                + 4 * (2 * len(new) + 1), "flops": 4 * case["hq"] * case["d"] * pairs}
    if case["op"] == "verify":
        elt = 4 if case["probs"] == "f32" else 2
        rows = case["batch"] * (2 if case["has_q"] else 1)
        counts = _draft_counts(case)
        return {"bytes": rows * case["vocab"] * elt + sum(counts) * (4 + 4 + 2 * elt)
                + case["batch"] * (4 + 4 + 4 + 4 * (case["drafts"] + 1)),
                "flops": 3 * rows * case["vocab"]}
    if case["op"] == "gather":
        first, count = _gather_ranges(case)
        elt = 1 if case["cache"] == "e4m3" else 2
        values = 2 * sum(count) * case["hkv"] * case["d"]
        return {"bytes": values * (elt + 2) + 8 * len(count)
                + 4 * sum((f + n - 1) // case["bs"] - f // case["bs"] + 1 for f, n in zip(first, count)),
                "flops": values if elt == 1 else 0}
    values = 2 * case["tokens"] * case["hkv"] * case["d"]
    return {"bytes": 2 * values + 8 * case["tokens"] + 2 * 16 * case["hkv"] * case["d"], "flops": values}


# ---- the definitions, in 64 bits ----------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "verify":  # whole numbers
        return None
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _attend_exact(case, s)
    if case["op"] == "gather":
        first, count = _gather_ranges(case)
        out, at = {"k": s["k_out"].double(), "v": s["v_out"].double()}, 0
        for b, (f, n) in enumerate(zip(first, count)):
            for name, w in (("k", 0), ("v", 1)):
                out[name][at:at + n] = _sequence(case, s, name + "_cache", w, b, f + n)[f:]
            at += n
        return out
    out = {}
    for name in ("k", "v"):
        x = s[name][s["slots"] >= 0].double().abs()
        x[~torch.isfinite(x)] = 0.0
        amax = torch.cat([s[name + "_amax"].double()[None], x]).max(0).values
        scale = (amax / E4M3_MAX).clamp(min=SMALLEST_SCALE)
        scale[amax == 0] = 1.0
        out[name + "_amax"], out[name + "_scale"], out[name + "_inv_scale"] = amax, scale, scale.reciprocal()
    return out


def _sequence(case, s, pool, which, b, length):
    """The first `length` cached rows of sequence b, block by block, in float64."""
    blocks = s["tables"][b, :-(-length // case["bs"])].long()
    rows = s[pool].index_select(0, blocks).flatten(0, 1)[:length]
    if s["scales"] is None:
        return rows.double()
    return rows.view(torch.float8_e4m3fn).to(torch.float64) * s["scales"][which].double()


def _attend_exact(case, s):
    new, ctx = _attend_lengths(case)
    group = case["hq"] // case["hkv"]
    out, at = s["out"].double(), 0
    for b, (n, L) in enumerate(zip(new, ctx)):
        k, v = (_sequence(case, s, x + "_cache", w, b, L) for w, x in enumerate("kv"))
        back = torch.arange(L - n, L, device=out.device)[:, None] - torch.arange(L, device=out.device)
        off = back < 0
        if case["window"]:
            off |= back >= case["window"]
        for h in range(case["hq"]):
            x = s["q"][at:at + n, h].double() @ k[:, h // group].T / math.sqrt(case["d"])
            out[at:at + n, h] = torch.softmax(x.masked_fill_(off, -math.inf), -1) @ v[:, h // group]
        at += n
    return out
