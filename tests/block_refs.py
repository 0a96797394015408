"""Plain 64-bit references of the 8-bit serving step (test-only): tables of a step, append with
block scales, attention over codes, verification of drafts.  Everything is written from the
definitions, on the CPU; inputs are CPU tensors."""
from __future__ import annotations

import math

import torch

E4M3 = torch.float8_e4m3fn
MOST = {"int8": 127, "e4m3": 448}
# half a step of a rounding, relative to the value
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def tables(ctx, new, counts, free, count, table, ps, max_tokens):
    """(table, free, count, counts, seq, qsl, slots, positions) of a step that fits."""
    table, free, counts = table.clone(), free.clone(), list(counts)
    stack = free[:count].tolist()
    for b, n in enumerate(new):
        if n < 0:
            stack += table[b, :counts[b]].tolist()
    seq, qsl, slots, pos = [], [0], [], []
    for b, n in enumerate(new):
        if n < 0:
            counts[b] = 0
        L = 0 if n < 0 else ctx[b] + n
        seq.append(L)
        qsl.append(qsl[-1] + max(n, 0))
        while n >= 0 and counts[b] * ps < L:
            table[b, counts[b]] = stack.pop()
            counts[b] += 1
        for p in range(ctx[b], L):
            slots.append(int(table[b, p // ps]) * ps + p % ps)
            pos.append(p)
    free[:len(stack)] = torch.tensor(stack, dtype=torch.int32)
    pad = max_tokens - len(slots)
    return table, free, len(stack), counts, seq, qsl, slots + [-1] * pad, pos + [0] * pad


def values(codes):
    """The numbers codes are, in float64 (uint8: e4m3)."""
    return codes.double() if codes.dtype == torch.int8 else codes.view(E4M3).float().double()


def grid_of(kind):
    if kind == "int8":
        return torch.arange(-127, 128).double()
    x = torch.arange(256).to(torch.uint8).view(E4M3).float().double()
    return x[x.isfinite()].unique()


def nearest(kind, x):
    """The code value next to x (float64), of two the even one; beyond the ends the end."""
    grid = grid_of(kind)
    k = torch.searchsorted(grid, x.clamp(float(grid[0]), float(grid[-1])).contiguous()).clamp(1, grid.numel() - 1)
    lo, hi = grid[k - 1], grid[k]
    low_even = torch.remainder(lo / (hi - lo), 2) == 0
    up = (x - lo > hi - x) | ((x - lo == hi - x) & ~low_even)
    return torch.where(up, hi, lo)


def append(kind, x, cache, scales, table, seq, qsl, ps):
    """(values, scales) of one cache (K or V) after the append of the packed rows x [T, H, D] (bf16)."""
    v, scales = values(cache), scales.clone()
    x = x.double()
    for b, L in enumerate(seq):
        n = qsl[b + 1] - qsl[b]
        if n == 0:
            continue
        ctx = L - n
        for i in range(ctx // ps, -(-L // ps)):
            page = int(table[b, i])
            kept, end = max(0, ctx - i * ps), min(ps, L - i * ps)
            rows = x[qsl[b] + i * ps + kept - ctx:qsl[b] + i * ps + end - ctx]
            fin = torch.where(rows.isfinite(), rows, 0.0)
            scale = (fin.abs().amax((0, 2)) / MOST[kind]).float()
            if kept:
                was = scales[page].clone()
                scale = torch.maximum(scale, was)
                for h in (scale > was).nonzero().flatten().tolist():
                    v[page, :kept, h] = nearest(kind, v[page, :kept, h] * was[h].double() / scale[h].double())
            scales[page] = scale
            q = rows / torch.where(scale > 0, scale, torch.ones_like(scale)).double()[:, None]
            code = nearest(kind, torch.where(rows.isnan(), 0.0, q))
            v[page, kept:end] = torch.where(rows.isnan(), 0.0 if kind == "int8" else math.nan, code)
    return v, scales


def attend(q, kc, vc, ks, vs, table, seq, qsl, scale, window=0, sinks=None, cap=0.0, chunked=False):
    """(out, lse, bounds of both) in float64 for packed rows (qsl None: one row a request).  The bounds are those of
    the kernels' roundings: a weight in f16 (half a step, relative; and where it is subnormal half of f16's least step,
    2^-25, which with weights of up to 2^14 -- 2^7 in chunks -- is 2^-39 -- 2^-32 -- of the row's largest weight times
    V scale, for each code it meets), fp32 sums of D products and of n keys (a step of 2^-23 for each addition),
    exponentials and logarithms good to 2^-20, and the output in bf16."""
    T, Hq, D = q.shape
    pool, ps, Hkv = kc.shape[0], kc.shape[1], kc.shape[2]
    G = Hq // Hkv
    out, lse = torch.zeros(T, Hq, D, dtype=torch.float64), torch.full((T, Hq), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for b, L in enumerate(seq):
        begin, n = (b, 1) if qsl is None else (qsl[b], qsl[b + 1] - qsl[b])
        ids = [int(x) for x in table[b, :-(-L // ps)]]
        for h in range(Hkv):
            rows = slice(h * G, (h + 1) * G)
            if L == 0:
                if sinks is not None and n:
                    lse[begin:begin + n, rows] = sinks[rows].double()
                continue
            def load(cache, sc):
                parts = [values(cache[i, :, h].contiguous()) * sc[i, h].double() if 0 <= i < pool
                         else torch.zeros(ps, D, dtype=torch.float64) for i in ids]
                return torch.cat(parts)[:L]
            k, v = load(kc, ks), load(vc, vs)
            size_v = torch.tensor([float(vs[i, h]) if 0 <= i < pool else 0.0 for i in ids],
                                  dtype=torch.float64).repeat_interleave(ps)[:L].clamp(min=2.0 ** -100)
            for r in range(n):
                pos = L - n + r
                lo = max(0, pos - window + 1) if window else 0
                qq = q[begin + r, rows].double()
                x = qq @ k[lo:pos + 1].t() * scale
                size = float((qq.abs() @ k[lo:pos + 1].abs().t()).max()) * abs(scale)
                eps = 2.0 ** -23 * (D + 16) * size + 2.0 ** -20
                if cap:
                    x = cap * torch.tanh(x / cap)
                    eps += 2.0 ** -18 * cap      # tanh to a few units of 2^-23, by the cap
                eps += 2.0 ** -22 * float(x.abs().max())
                vv, sv = v[lo:pos + 1], size_v[lo:pos + 1]
                if sinks is not None:
                    x = torch.cat([x, sinks[rows, None].double()], 1)
                    vv = torch.cat([vv, torch.zeros(1, D, dtype=torch.float64)])
                w = torch.softmax(x, 1)
                out[begin + r, rows] = w @ vv
                lse[begin + r, rows] = torch.logsumexp(x, 1)
                keys = pos + 1 - lo
                rel = HALF["f16"] + 2 * eps + 2.0 ** -23 * keys
                keyed = w[:, :keys] * sv
                least = (2.0 ** -32 if chunked else 2.0 ** -39) * keyed.max(1, keepdim=True).values \
                    * (vv[:keys].abs() / sv[:, None]).sum(0)
                tol_o[begin + r, rows] = rel * (w @ vv.abs()) + least + HALF["bf16"] * out[begin + r, rows].abs() \
                    + 2.0 ** -100
                tol_l[begin + r, rows] = eps + 2.0 ** -23 * (keys + 16) + 2.0 ** -22 * lse[begin + r, rows].abs()
    return out, lse, tol_o, tol_l


def verify(tokens, p, q, qsl, u, w, width):
    """(out, num) of verify_tokens (q None: certain drafts)."""
    out, num = torch.full((len(qsl) - 1, width), -1, dtype=torch.int32), torch.zeros(len(qsl) - 1, dtype=torch.int32)

    def clean(x):
        return torch.where(x > 0, x, torch.zeros_like(x)).double()
    V = p.shape[1]
    for b in range(len(qsl) - 1):
        n = qsl[b + 1] - qsl[b]
        for i in range(n):
            r = qsl[b] + i
            pr = clean(p[r])
            y = pr
            if i < n - 1:
                x = int(tokens[r + 1])
                inside = 0 <= x < V
                qr = torch.zeros(V, dtype=torch.float64) if q is None else clean(q[r])
                if q is None and inside:
                    qr[x] = 1.0
                qx = 1.0 if q is None else (float(qr[x]) if inside else 0.0)
                if float(u[r]) * qx < (float(pr[x]) if inside else 0.0):
                    out[b, i] = x
                    continue
                y = (pr - qr).clamp(min=0)
                if not bool((y > 0).any()):
                    y = pr
            num[b] = i + 1
            if bool((y > 0).any()):
                c = y.cumsum(0)
                v = int(torch.searchsorted(c, float(w[b]) * c[-1], right=True))
                out[b, i] = min(v, int((y > 0).nonzero().max()))
            break
    return out, num
