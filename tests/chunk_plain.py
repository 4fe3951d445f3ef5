"""Plain forms, in 64 bits on the CPU, of the operators that serve chunks of
new tokens, and the bounds that their kernels' rounding may reach."""
import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # half a step, relative


def paged_rows(pool, scale, table, block_size, length):
    """The first `length` cached tokens of a block table in float64, token by token."""
    d = pool.view(torch.float8_e4m3fn).double() if pool.dtype == torch.uint8 else pool.double()
    if scale is not None:
        d = d * scale.double()
    out = torch.empty((length,) + tuple(pool.shape[2:]), dtype=torch.float64)
    for j in range(length):
        out[j] = d[int(table[j // block_size]), j % block_size]
    return out


def attend_chunk(q, k_pool, v_pool, cu, tables, lens, scale, out, window=0, k_scale=None,
                 v_scale=None):
    """(out, bound): float64 attention of each row over the tokens it sees, row by row, in a copy
    of `out`; `bound` is how far the kernel's rounding may take each value from it:
      - P and, at the end, the result are rounded to the operands' 16 bits: u sum_j w_j |v_j|
        and u |out|;
      - the scores are 32-bit sums (each step of 16 products rounded or cut to 2^-23): their
        error moves the weights by at most twice itself;
      - an E4M3 cache's q * k_scale is rounded to f16: 2^-11 of each product of the score;
      - the 32-bit sum over tokens: one rounding of 2^-23 per 16 tokens; ex2.approx and the
        division: 2^-21."""
    hq, hkv = q.shape[1], k_pool.shape[2]
    bs, d = k_pool.shape[1], q.shape[2]
    group = hq // hkv
    res = out.double().clone()
    bound = torch.zeros_like(res)
    u = U[q.dtype]
    up = U[torch.float16] if k_pool.dtype == torch.uint8 else u
    for b in range(len(lens)):
        n = int(cu[b + 1]) - int(cu[b])
        L = int(lens[b])
        if n == 0:
            continue
        k = paged_rows(k_pool, k_scale, tables[b], bs, L)
        v = paged_rows(v_pool, v_scale, tables[b], bs, L)
        for i in range(n):
            r, pos = int(cu[b]) + i, L - n + i
            lo = max(0, pos - window + 1) if window else 0
            for h in range(hq):
                kk, vv = k[lo:pos + 1, h // group], v[lo:pos + 1, h // group]
                s = kk @ q[r, h].double() * scale
                w = torch.softmax(s, 0)
                o = w @ vv
                size = float((kk.abs() @ q[r, h].double().abs()).max()) * abs(scale)
                e_s = size * (d / 16 + 16) * 2.0 ** -23
                if k_pool.dtype == torch.uint8:
                    e_s += size * 2.0 ** -11
                sums = ((pos + 1 - lo) / 16 + 16) * 2.0 ** -23
                a = w @ vv.abs()
                res[r, h] = o
                bound[r, h] = a * (up + 2 * e_s + sums + 2.0 ** -21) + u * o.abs() + 2.0 ** -24
    return res, bound


def chunk_case(batch, hq, hkv, d, bs, dtype, chunks, ctxs, cache="io", pad=0, seed=0, junk=True):
    """Inputs on the CPU. Everything the rows may not see (unused blocks, rows behind a context)
    holds NaN (or, in an E4M3 cache, its NaN code), and unused table entries are out of range."""
    g = torch.Generator().manual_seed(1000 + seed)
    need = [-(-c // bs) for c in ctxs]
    nb = sum(need) + 3
    perm = torch.randperm(nb, generator=g).tolist()
    mb = max(1, max(need)) + 1
    tables = torch.full((batch, mb), 1 << 30 if junk else 0, dtype=torch.int32)
    shape = (nb, bs, hkv, d)
    live = torch.zeros(nb, bs, dtype=torch.bool)
    at = 0
    for b, m in enumerate(need):
        tables[b, :m] = torch.tensor(perm[at:at + m], dtype=torch.int32)
        for j in range(ctxs[b]):
            live[perm[at + j // bs], j % bs] = True
        at += m
    c = {"scales": None}
    for name in ("k", "v"):
        x = torch.randn(shape, generator=g)
        if cache == "e4m3":
            codes = (x * 90).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            if junk:
                codes[~live] = 0x7f
            c[name] = codes
            c[name + "_scale"] = (torch.rand((hkv, d), generator=g) * 1.5 + 0.5) / 90
        else:
            x = x.to(dtype)
            if junk:
                x[~live] = float("nan")
            c[name] = x
            c[name + "_scale"] = None
    cu = [0]
    for n in chunks:
        cu.append(cu[-1] + n)
    c["cu"] = torch.tensor(cu, dtype=torch.int32)
    c["lens"] = torch.tensor(ctxs, dtype=torch.int32)
    c["tables"] = tables
    rows = cu[-1] + pad
    c["q"] = torch.randn((rows, hq, d), generator=g).to(dtype)
    c["out"] = torch.randn((rows, hq, d), generator=g).to(dtype)
    c["scale"] = 1 / math.sqrt(d)
    c["max_chunk"], c["max_context"] = max(chunks), max(ctxs)
    return c


def on_gpu(c, device="cuda"):
    return {k: v.to(device) if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def weight(x):
    """A probability row in float64; what is not positive and finite counts as zero."""
    x = x.double()
    return torch.where((x > 0) & (x < math.inf), x, 0.0)


def verify_draft(drafts, cu, target, draft, u_accept, u_sample, most):
    """(accepted, tokens) by the definition, one sequence at a time."""
    accepted, rows = [], []
    for b in range(len(cu) - 1):
        start, n = int(cu[b]), int(cu[b + 1]) - int(cu[b])
        a = 0
        while a < n:
            x = int(drafts[start + a])
            if not 0 <= x < target.shape[1]:
                break
            p = float(weight(target[start + b + a, x]))
            q = 1.0 if draft is None else float(weight(draft[start + a, x]))
            if not float(u_accept[start + a].double()) * q < p:
                break
            a += 1
        p = weight(target[start + b + a])
        w = p.clone()
        if a < n:
            if draft is None:
                if 0 <= int(drafts[start + a]) < len(w):
                    w[int(drafts[start + a])] = 0.0
            else:
                w = (p - weight(draft[start + a])).clamp(min=0.0)
            if float(w.sum()) == 0.0:
                w = p
        token = -1
        total = math.fsum(w.tolist())
        if total > 0:
            run = torch.cumsum(w, 0)
            past = ((run > float(u_sample[b].double()) * total) & (w > 0)).nonzero()
            token = int(past[0]) if len(past) else int((w > 0).nonzero()[-1])
        accepted.append(a)
        rows.append([int(drafts[start + i]) for i in range(a)] + [token] + [-1] * (most - a))
    return accepted, rows


def calibrate(x, slots, amax):
    """(amax, scale, inv_scale) in float32, by the definition."""
    x = x.double().abs()
    x = torch.where(torch.isfinite(x), x, 0.0)
    if slots is not None:
        x = x[slots >= 0]
    amax = torch.cat([amax.double()[None], x]).amax(0).float()
    scale = (amax / 448.0).clamp(min=2.0 ** -126)
    scale = torch.where(amax > 0, scale, 1.0)
    return amax, scale, 1.0 / scale
