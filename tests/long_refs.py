"""Plain 64-bit references of the long-context operators (test-only): norm and
rotation, key bounds of pages, page selection, attention over chosen pages.
Everything is written from the definitions, one row and head at a time, on the
CPU; inputs are CPU tensors."""
from __future__ import annotations

import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}


def kv_values(codes, scale):
    """Cache elements as float64: bf16 as they are, e4m3 codes as bf16(code * scale)."""
    if codes.dtype == torch.uint8:
        x = codes.view(torch.float8_e4m3fn).float() * torch.tensor(scale, dtype=torch.float32)
        return x.to(torch.bfloat16).double()
    return codes.double()


def norm_rotate(x, w, positions, table, *, rot, interleaved, sections, eps, offset):
    """(y, m): y the normed and rotated rows of x [T, H, D], m [T, H, D] the length of each element's pair."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (w.double() + offset)
    y, m = x.clone(), x.abs()
    half = rot // 2
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    for i in range(half):
        p = positions[axis[i]].long().clamp(0, table.shape[0] - 1)      # (tokens with another one are not written)
        cos, sin = table.double()[p, i][:, None], table.double()[p, half + i][:, None]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., b] * cos + x[..., a] * sin
        m[..., a] = m[..., b] = torch.hypot(x[..., a], x[..., b])
    return y, m


def bounds_of(k_cache, block_table, seq_lens, page_size, scale=1.0, scales=None):
    """{pool page: [Hkv, 2, D]} of every page of every request (float64)."""
    out = {}
    for b, L in enumerate(seq_lens):
        for i in range(-(-L // page_size)):
            page = int(block_table[b, i])
            k = kv_values(k_cache[page, :min(page_size, L - i * page_size)], scale if scales is None else float(scales[b]))
            out[page] = torch.stack([k.min(0).values, k.max(0).values], 1)
    return out


def rows_of(seq_lens, query_start_loc=None):
    """[(row, request, position)] of every query row."""
    if query_start_loc is None:
        return [(b, b, L - 1) for b, L in enumerate(seq_lens)]
    out = []
    for b, L in enumerate(seq_lens):
        n = query_start_loc[b + 1] - query_start_loc[b]
        out += [(query_start_loc[b] + i, b, L - n + i) for i in range(n)]
    return out


def page_scores(q, bounds, block_table, b, kvh, n):
    """Exact scores [n] of the first n pages for the heads q [G, D] of a row."""
    best = None
    rows = bounds[block_table[b, :n].long(), kvh].double()          # [n, 2, D]
    odd = ~torch.isfinite(rows).all(-1).all(-1)
    for x in q.double():
        lo, hi = x * rows[:, 0], x * rows[:, 1]
        u = torch.where(x == 0, torch.zeros_like(lo), torch.maximum(lo, hi)).sum(-1)
        u = torch.where(torch.isfinite(u) & ~odd & torch.isfinite(x).all(), u, torch.full_like(u, math.inf))
        best = u if best is None else torch.maximum(best, u)
    return best


def select(q, bounds, block_table, seq_lens, *, page_size, num_kv_heads, top, first, last, query_start_loc=None):
    """{row: [Hkv, top] chosen pages, ascending, then -1}."""
    G = q.shape[1] // num_kv_heads
    out = {}
    for row, b, pos in rows_of(seq_lens, query_start_loc):
        n = pos // page_size + 1 if pos >= 0 else 0
        r = torch.full((num_kv_heads, top), -1, dtype=torch.int32)
        for h in range(num_kv_heads):
            if n <= top:
                pick = list(range(n))
            else:
                s = page_scores(q[row, h * G:(h + 1) * G], bounds, block_table, b, h, n).tolist()
                free = sorted(range(first, n - last), key=lambda i: (-s[i], i))[:top - first - last]
                pick = sorted(list(range(first)) + free + list(range(n - last, n)))
            r[h, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
        out[row] = r
    return out


def attend(q, k_cache, v_cache, block_table, seq_lens, pages, *, page_size, scale, query_start_loc=None, sinks=None,
           soft_cap=0.0, k_scale=1.0, v_scale=1.0, k_scales=None, v_scales=None):
    """{row: (out [Hq, D], lse [Hq], spread [Hq, D])}; spread = sum of weight * |value|."""
    Hkv, D = k_cache.shape[2], k_cache.shape[3]
    G = q.shape[1] // Hkv
    res = {}
    for row, b, pos in rows_of(seq_lens, query_start_loc):
        o = torch.zeros(Hkv * G, D, dtype=torch.float64)
        spread = torch.zeros_like(o)
        lse = torch.full((Hkv * G,), -math.inf, dtype=torch.float64)
        for h in range(Hkv):
            ks, vs = [], []
            for page in pages[row, h].tolist():
                if page < 0:
                    continue
                there = min(page_size, pos + 1 - page * page_size)
                if there <= 0:
                    continue
                pool = int(block_table[b, page])
                ks.append(kv_values(k_cache[pool, :there, h], k_scale if k_scales is None else float(k_scales[b])))
                vs.append(kv_values(v_cache[pool, :there, h], v_scale if v_scales is None else float(v_scales[b])))
            k = torch.cat(ks) if ks else torch.zeros(0, D, dtype=torch.float64)
            v = torch.cat(vs) if vs else torch.zeros(0, D, dtype=torch.float64)
            for j in range(h * G, (h + 1) * G):
                s = (k @ q[row, j].double()) * scale
                if soft_cap > 0:
                    s = soft_cap * torch.tanh(s / soft_cap)
                if sinks is not None:
                    s = torch.cat([s, sinks[j:j + 1].double()])
                if s.numel() == 0:
                    continue
                lse[j] = torch.logsumexp(s, 0)
                w = torch.exp(s - lse[j])[:k.shape[0]]
                o[j], spread[j] = w @ v, w @ v.abs()
        res[row] = (o, lse, spread)
    return res


def attend_tolerance(o, spread):
    """Half a bf16 step of the output; a bf16 rounding of every weight (2^-8 of it, at most: weights that carry a row
    are held to 2^-17); 2^-11 for the 32-bit scores: D <= 256 additions, each off by 2^-24 of sum |q k| scale (at most
    about 11 for these inputs), are below 2^-12 in the exponent, once in the weight and once in the denominator."""
    return 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -11) * spread + 1e-30
