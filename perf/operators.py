"""The serving step over a long paged context, operator by operator.

A step of a model with a long context calls, per layer: the append of the new
tokens' keys and values (norm and rotation of queries and keys on the way),
the refresh of the key bounds of the pages written, the selection of the pages
each query attends to, and the attention over those pages.  Each case is one
of the four; ``run`` computes it with elementary torch operations, or, where
``own`` is true, by the calls of ``paged_kv_gqa_12_gb300.binding``.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------

def _append(name, tokens, q_heads, kv_heads, dim, page, kv="bf16", norm=False, axes=1, rot=None, interleaved=False):
    return dict(name=name, op="append", tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, dim=dim, page=page, kv=kv,
                norm=norm, axes=axes, rot=dim if rot is None else rot, interleaved=interleaved)


def _bounds(name, batch, len_lo, len_hi, new, kv_heads, dim, page, kv="bf16"):
    return dict(name=name, op="bounds", batch=batch, len_lo=len_lo, len_hi=len_hi, new=new, kv_heads=kv_heads, dim=dim,
                page=page, kv=kv)


def _select(name, batch, len_lo, len_hi, new, q_heads, kv_heads, dim, page, top, first=1, last=2):
    return dict(name=name, op="select", batch=batch, len_lo=len_lo, len_hi=len_hi, new=new, q_heads=q_heads,
                kv_heads=kv_heads, dim=dim, page=page, top=top, first=first, last=last)


def _attend(name, batch, len_lo, len_hi, new, q_heads, kv_heads, dim, page, top, first=1, last=2, kv="bf16", sinks=False,
            cap=0.0):
    return dict(name=name, op="attend", batch=batch, len_lo=len_lo, len_hi=len_hi, new=new, q_heads=q_heads,
                kv_heads=kv_heads, dim=dim, page=page, top=top, first=first, last=last, kv=kv, sinks=sinks, cap=cap)


def listed():
    return [
        # a decode step of four requests of a small model: latency alone
        _append("append_decode_4", 4, 8, 2, 64, 16),
        # a decode step of 250 requests, per-head norms, into an e4m3 cache
        _append("append_decode_250_e4m3", 250, 32, 8, 128, 64, kv="e4m3", norm=True),
        # a prefill step of packed text and image tokens: three position axes, per-head norms
        _append("append_prefill_16381", 16381, 32, 8, 128, 16, norm=True, axes=3),
        # a decode step: each of 64 requests has one page that changed
        _bounds("bounds_decode_64", 64, 512, 8192, 1, 8, 128, 16),
        # chunks of new tokens of 32 requests in an e4m3 cache
        _bounds("bounds_chunk_32_e4m3", 32, 2048, 32768, 2000, 8, 64, 64, kv="e4m3"),
        # whole contexts of 8 requests, as after loading a cached prefix
        _bounds("bounds_whole_8", 8, 8192, 32768, 0, 8, 128, 16),
        # one request deep in a context of 131071 tokens
        _select("select_one_131071", 1, 131071, 131071, 1, 32, 8, 128, 16, 128, last=4),
        # a decode step of 64 requests
        _select("select_decode_64", 64, 4096, 32768, 1, 32, 8, 128, 16, 128, last=4),
        # chunks of new tokens of 4 requests, 8 heads a kv head
        _select("select_chunk_4", 4, 8192, 32768, 160, 64, 8, 64, 64, 32),
        # four short requests of a small model
        _attend("attend_decode_4", 4, 60, 1000, 1, 8, 2, 64, 16, 16),
        # a decode step of 64 requests, 2048 keys each
        _attend("attend_decode_64", 64, 4096, 32768, 1, 32, 8, 128, 16, 128, last=4),
        # chunks of new tokens of 4 requests over an e4m3 cache, with sinks
        _attend("attend_chunk_4_e4m3", 4, 8192, 32768, 160, 64, 8, 64, 64, 32, kv="e4m3", sinks=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# (q heads, kv heads, head dim): the small, the Llama-3-8B-shaped, the wide and the head_dim-256 ones, and odd groups
_HEADS = [(8, 2, 64), (32, 8, 128), (64, 8, 64), (16, 8, 256), (24, 8, 128), (28, 4, 128), (8, 8, 64), (40, 2, 128)]


def draw(rng):
    """A case of the listed ones' ranges that costs no more than the largest listed one of its operator."""
    while True:
        case = _draw(rng)
        most = [work(c) for c in listed() if c["op"] == case["op"]]
        if all(v <= max(w[k] for w in most) for k, v in work(case).items()):
            return case


def _draw(rng):
    op = rng.choice(["append", "bounds", "select", "attend"])
    hq, hkv, dim = rng.choice(_HEADS)
    page = rng.choice([16, 32, 64])
    kv = rng.choice(["bf16", "e4m3"])
    if op == "append":
        rot = rng.choice([dim, dim, dim // 2])
        c = _append("", _log_uniform(rng, 1, 8000), hq, hkv, dim, page, kv=kv, norm=rng.random() < 0.5,
                    axes=rng.choice([1, 1, 3]), rot=rot, interleaved=rng.random() < 0.3)
    else:
        batch = _log_uniform(rng, 1, 64)
        # contexts of at most 400,000 tokens in all; a selection is for long ones
        hi = _log_uniform(rng, 100 if op == "bounds" else 2000, min(131071, 400000 // batch))
        lo = max(1, int(hi * rng.uniform(0.05, 1.0)))
        if op == "bounds":
            new = rng.choice([0, 1, _log_uniform(rng, 2, 2000)])
            c = _bounds("", batch, lo, hi, min(new, lo), hkv, dim, page, kv=kv)
        else:
            # at most about 300 query rows; up to half of the longest context, so short ones are attended whole
            new = min(lo, rng.choice([1, 1, _log_uniform(rng, 2, max(2, 300 // batch))]))
            first, last = rng.randint(0, 2), rng.randint(1, 4)
            keys = _log_uniform(rng, min(8 * page, hi // 4), min(2048, hi // 2))
            top = max(first + last, keys // page)
            if op == "select":
                c = _select("", batch, lo, hi, new, hq, hkv, dim, page, top, first, last)
            else:
                c = _attend("", batch, lo, hi, new, hq, hkv, dim, page, top, first, last, kv=kv,
                            sinks=rng.random() < 0.3, cap=rng.choice([0.0, 0.0, 30.0]))
    del c["name"]
    return c


# ---- inputs --------------------------------------------------------------------

def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]: the same for every seed, so that the work of a case is known."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lens(case):
    return _spread(case["len_lo"], case["len_hi"], case["batch"])


def _rows(case):
    """New tokens of each request, in the order of _lens."""
    n = case["new"]
    if n <= 1:
        return [1] * case["batch"]
    return _spread(max(1, n // 4), n, case["batch"])


def _cdiv(a, b):
    return -(-a // b)


def _randn_bf16(shape, g):
    """N(0, 1) in bf16, made in pieces: a large pool never holds its 32-bit form whole."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda")
    return out


def _cache(shape, kv, scale, g):
    x = _randn_bf16(shape, g)
    if kv == "bf16":
        return x
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for a, b in zip(x.split(4096), out.split(4096)):
        b.copy_((a.float() / scale).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8))
    return out


def _paged(case, g):
    """Lengths (and new tokens) in a seeded order, and block tables over a shuffled pool."""
    B, ps = case["batch"], case["page"]
    order = torch.randperm(B, generator=g, device="cuda").tolist()
    lens = [_lens(case)[i] for i in order]
    rows = [_rows(case)[i] for i in order]
    n_pages = [_cdiv(L, ps) for L in lens]
    pool = sum(n_pages) + max(1, sum(n_pages) // 20)
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    W = max(n_pages)
    table = torch.zeros(B, W, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(n_pages):
        table[b, :n] = perm[at:at + n]
        at += n
    qsl = [0]
    for r in rows:
        qsl.append(qsl[-1] + r)
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(lens=lens, rows=rows, pool=pool, width=W, table=table, seq_lens=torch.tensor(lens, **i32),
                qsl=torch.tensor(qsl, **i32), total_q=qsl[-1], max_rows=max(rows))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    s = dict(case)
    return {"append": _prepare_append, "bounds": _prepare_bounds, "select": _prepare_select,
            "attend": _prepare_attend}[case["op"]](s, g)


def _prepare_append(s, g):
    T, Hq, Hkv, D, ps = s["tokens"], s["q_heads"], s["kv_heads"], s["dim"], s["page"]
    pool = _cdiv(T, ps) + 8
    # q, k and v are parts of one projection's output
    qkv = _randn_bf16((T, Hq + 2 * Hkv, D), g)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    s["slots"] = torch.randperm(pool * ps, generator=g, device="cuda")[:T].contiguous()
    max_pos = 65536
    pos = torch.randint(0, max_pos, (s["axes"], T), generator=g, device="cuda")
    s["positions"] = pos.to(torch.int32)
    rot = s["rot"]
    freq = 1e6 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    half = rot // 2
    # pairs of each axis: a quarter, and the rest in two (one axis: all)
    s["sections"] = (half,) if s["axes"] == 1 else (half // 4, half // 4 + half // 8, half - half // 2 - half // 8)
    axis = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
    s["axis_of_pair"] = torch.tensor(axis, device="cuda")
    s["wq"] = s["wk"] = None
    if s["norm"]:
        s["wq"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16()
        s["wk"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16()
    s["scale_k"], s["scale_v"] = (0.05, 0.04) if s["kv"] == "e4m3" else (1.0, 1.0)
    s["k_cache"] = _cache((pool, ps, Hkv, D), s["kv"], s["scale_k"], g)
    s["v_cache"] = _cache((pool, ps, Hkv, D), s["kv"], s["scale_v"], g)
    s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    if own:
        from paged_kv_gqa_12_gb300 import binding as pb
        s["rope"] = pb.rope(s["cos_sin"], rot_dim=rot, interleaved=s["interleaved"],
                            sections=None if s["axes"] == 1 else s["sections"], q_norm=s["wq"], k_norm=s["wk"],
                            norm_eps=EPS)
    return s


def _prepare_bounds(s, g):
    s.update(_paged(s, g))
    Hkv, D, ps = s["kv_heads"], s["dim"], s["page"]
    s["scale_k"] = 0.05 if s["kv"] == "e4m3" else 1.0
    s["k_cache"] = _cache((s["pool"], ps, Hkv, D), s["kv"], s["scale_k"], g)
    s["bounds"] = torch.zeros(s["pool"], Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    # pages a request can have changed: its new tokens' pages, or all
    s["most"] = max(_cdiv(L, ps) - (L - r) // ps for L, r in zip(s["lens"], s["rows"])) if s["new"] else s["width"]
    return s


def _sparse_plan(s, kv):
    from paged_kv_gqa_12_gb300 import binding as pb
    s["plan"] = pb.sparse_plan(num_q_heads=s["q_heads"], num_kv_heads=s["kv_heads"], head_dim=s["dim"],
                               page_size=s["page"], kv_dtype=pb.KV_FP8_E4M3 if kv == "e4m3" else pb.KV_BF16,
                               max_batch=s["batch"], max_pages_per_seq=s["width"], max_total_q=s["total_q"],
                               top_pages=s["top"], first_pages=s["first"], last_pages=s["last"],
                               has_sinks=bool(s.get("sinks")), soft_cap=s.get("cap", 0.0))
    s["scratch"] = pb.alloc_scratch(s["plan"])


def _prepare_select(s, g):
    s.update(_paged(s, g))
    Hkv, D, ps = s["kv_heads"], s["dim"], s["page"]
    s["q"] = _randn_bf16((s["total_q"], s["q_heads"], D), g)
    s["bounds"] = torch.empty(s["pool"], Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    for part in s["bounds"].split(1024):
        # keys of a page lie around a direction of the page's own
        k = torch.randn(part.shape[0], ps, Hkv, D, generator=g, device="cuda")
        k = (k + torch.randn(part.shape[0], 1, Hkv, D, generator=g, device="cuda")) * 0.7
        part[:, :, 0] = k.amin(1)
        part[:, :, 1] = k.amax(1)
    s["pages"] = torch.empty(s["total_q"], Hkv, s["top"], dtype=torch.int32, device="cuda")
    if own:
        _sparse_plan(s, "bf16")
    return s


def _prepare_attend(s, g):
    s.update(_paged(s, g))
    Hq, Hkv, D, ps, T = s["q_heads"], s["kv_heads"], s["dim"], s["page"], s["total_q"]
    s["q"] = _randn_bf16((T, Hq, D), g)
    s["scale_k"], s["scale_v"] = (0.05, 0.04) if s["kv"] == "e4m3" else (1.0, 1.0)
    s["k_cache"] = _cache((s["pool"], ps, Hkv, D), s["kv"], s["scale_k"], g)
    s["v_cache"] = _cache((s["pool"], ps, Hkv, D), s["kv"], s["scale_v"], g)
    n = _row_places(s)[1].div(ps, rounding_mode="floor") + 1
    s["pages"] = _best_pages(s, torch.rand(T, Hkv, s["width"], generator=g, device="cuda"), n).contiguous()
    s["sink"] = torch.randn(Hq, generator=g, device="cuda") if s["sinks"] else None
    s["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(T, Hq, dtype=torch.float32, device="cuda")
    if own:
        _sparse_plan(s, s["kv"])
    return s


# ---- one pass ------------------------------------------------------------------

def run(s):
    return {"append": _run_append, "bounds": _run_bounds, "select": _run_select, "attend": _run_attend}[s["op"]](s)


def _kv_type(s):
    from paged_kv_gqa_12_gb300 import binding as pb
    return pb.KV_FP8_E4M3 if s["kv"] == "e4m3" else pb.KV_BF16


def _values(cache):
    """A cache as the values it holds: e4m3 codes as e4m3 numbers."""
    return cache.view(E4M3) if cache.dtype == torch.uint8 else cache


def _norm_rotate(s, x, w):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    rot, half = s["rot"], s["rot"] // 2
    pair = torch.arange(half, device="cuda")
    at = s["positions"].long()[s["axis_of_pair"]].t()            # [T, half]: each pair's position
    cos, sin = s["cos_sin"][at, pair][:, None], s["cos_sin"][at, half + pair][:, None]
    if s["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _run_append(s):
    if own:
        from paged_kv_gqa_12_gb300 import binding as pb
        pb.append_rope_kv(s["rope"], s["k"], s["v"], s["positions"], s["k_cache"], s["v_cache"], s["slots"], q=s["q"],
                          q_out=s["q_out"], kv_dtype=_kv_type(s), k_scale=s["scale_k"], v_scale=s["scale_v"])
        return s["q_out"], _values(s["k_cache"]), _values(s["v_cache"])
    s["q_out"].copy_(_norm_rotate(s, s["q"], s["wq"]))
    k, v = _norm_rotate(s, s["k"], s["wk"]), s["v"]
    if s["kv"] == "e4m3":
        k = (k / s["scale_k"]).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
        v = (v.float() / s["scale_v"]).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
    ps, Hkv, D = s["page"], s["kv_heads"], s["dim"]
    s["k_cache"].view(-1, Hkv, D)[s["slots"]] = k.to(s["k_cache"].dtype)
    s["v_cache"].view(-1, Hkv, D)[s["slots"]] = v.to(s["v_cache"].dtype)
    return s["q_out"], _values(s["k_cache"]), _values(s["v_cache"])


def _keys(s, codes, scale):
    """A cache's elements as numbers: e4m3 dequantises to bf16(code * scale)."""
    if s["kv"] == "e4m3":
        return (codes.view(E4M3).float() * scale).bfloat16().float()
    return codes.float()


def _run_bounds(s):
    if own:
        from paged_kv_gqa_12_gb300 import binding as pb
        pb.page_bounds(s["k_cache"], s["table"], s["seq_lens"], s["bounds"],
                       query_start_loc=s["qsl"] if s["new"] else None, kv_dtype=_kv_type(s), k_scale=s["scale_k"])
        return s["bounds"]
    ps, L = s["page"], s["seq_lens"].long()
    new = (s["qsl"][1:] - s["qsl"][:-1]).long() if s["new"] else L
    first, last = (L - new) // ps, (L - 1) // ps
    i = torch.minimum(first[:, None] + torch.arange(s["most"], device="cuda"), last[:, None])   # [B, most]
    ids = torch.gather(s["table"].long(), 1, i)
    k = _keys(s, s["k_cache"][ids], s["scale_k"])                                      # [B, most, ps, Hkv, D]
    there = (i[..., None] * ps + torch.arange(ps, device="cuda") < L[:, None, None])[..., None, None]
    s["bounds"][ids, :, 0] = k.masked_fill(~there, math.inf).amin(2).bfloat16()
    s["bounds"][ids, :, 1] = k.masked_fill(~there, -math.inf).amax(2).bfloat16()
    return s["bounds"]


def _row_places(s):
    """(request, position) of every query row."""
    row = torch.arange(s["total_q"], device="cuda")
    req = torch.searchsorted(s["qsl"].long(), row, right=True) - 1
    return req, s["seq_lens"].long()[req] - s["qsl"].long()[req + 1] + row


def _best_pages(s, score, n):
    """The pages of each row (of n visible ones) and kv head, ascending, -1 behind the last: the first and the last
    pages, then the highest scores; ties go to the lowest page."""
    W, top = score.shape[-1], s["top"]
    page = torch.arange(W, device="cuda")
    n = n[:, None, None]
    forced = (page < s["first"]) | (page >= n - s["last"])
    score = score.masked_fill(forced, math.inf).masked_fill(page >= n, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    rank = torch.arange(order.shape[-1], device="cuda")
    best = torch.sort(order.masked_fill(rank >= n, W), dim=-1).values
    best = best.masked_fill(best == W, -1)
    return torch.nn.functional.pad(best, (0, top - best.shape[-1]), value=-1).to(torch.int32)


def _run_select(s):
    if own:
        from paged_kv_gqa_12_gb300 import binding as pb
        pb.select_pages(s["plan"], s["q"], s["bounds"], s["table"], s["seq_lens"], s["pages"],
                        query_start_loc=s["qsl"] if s["new"] > 1 else None, scratch=s["scratch"])
        return s["pages"]
    Hkv, D, B, R = s["kv_heads"], s["dim"], s["batch"], s["max_rows"]
    req, pos = _row_places(s)
    # the order of two scores next to the border needs 64 bits
    b = s["bounds"][s["table"].long()].double()                  # [B, W, Hkv, 2, D]
    rows = (s["qsl"][:-1].long()[:, None] + torch.arange(R, device="cuda")).clamp(max=s["total_q"] - 1)
    q = s["q"][rows].double().reshape(B, R, Hkv, -1, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    b = b.permute(0, 2, 3, 4, 1)                                 # [B, Hkv, 2, D, W]
    u = q.clamp(max=0) @ b[:, :, 0] + q.clamp(min=0) @ b[:, :, 1]
    score = u.reshape(B, Hkv, R, -1, u.shape[-1]).amax(3).permute(0, 2, 1, 3)        # [B, R, Hkv, W]
    score = score[req, torch.arange(s["total_q"], device="cuda") - s["qsl"].long()[req]]
    s["pages"].copy_(_best_pages(s, score, pos.div(s["page"], rounding_mode="floor") + 1))
    return s["pages"]


def _run_attend(s):
    if own:
        from paged_kv_gqa_12_gb300 import binding as pb
        pb.sparse_attend(s["plan"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"], s["pages"],
                         query_start_loc=s["qsl"] if s["new"] > 1 else None, scale=s["dim"] ** -0.5, out=s["out"],
                         lse=s["lse"], sinks=s["sink"], k_scale=s["scale_k"], v_scale=s["scale_v"],
                         scratch=s["scratch"])
        return s["out"], s["lse"]
    T, Hkv, D, ps = s["total_q"], s["kv_heads"], s["dim"], s["page"]
    req, pos = _row_places(s)
    pages = s["pages"].long()
    ids = s["table"].long()[req[:, None, None], pages.clamp(min=0)]
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    k = _keys(s, s["k_cache"][ids, :, head], s["scale_k"]).reshape(T, Hkv, -1, D)
    v = _keys(s, s["v_cache"][ids, :, head], s["scale_v"]).reshape(T, Hkv, -1, D)
    at = pages[..., None] * ps + torch.arange(ps, device="cuda")
    seen = ((pages[..., None] >= 0) & (at <= pos[:, None, None, None])).reshape(T, Hkv, 1, -1)
    q = s["q"].float().reshape(T, Hkv, -1, D)
    x = (q @ k.transpose(-1, -2)) * D ** -0.5
    if s["cap"]:
        x = s["cap"] * torch.tanh(x / s["cap"])
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].reshape(1, Hkv, -1, 1)
        top = torch.maximum(top, sink)
    e = torch.exp(x - top)
    z = e.sum(-1, keepdim=True)
    if s["sink"] is not None:
        z = z + torch.exp(sink - top)
    s["out"].copy_(((e @ v) / z).reshape(T, -1, D))
    s["lse"].copy_((top + torch.log(z)).reshape(T, -1))
    return s["out"], s["lse"]


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    e = 1 if case.get("kv") == "e4m3" else 2
    D, ps = case["dim"], case["page"]
    if case["op"] == "append":
        T, Hq, Hkv = case["tokens"], case["q_heads"], case["kv_heads"]
        move = T * D * (2 * 2 * Hq + 2 * (2 + e) * Hkv)
        turn = T * case["axes"] * 4 + T * 8 + T * case["rot"] * 4
        return {"bytes": move + turn, "flops": T * (Hq + Hkv) * (3 * case["rot"] + (4 * D if case["norm"] else 0))}
    Hkv, lens, rows = case["kv_heads"], _lens(case), _rows(case)
    if case["op"] == "bounds":
        new = rows if case["new"] else lens
        pages = [_cdiv(L, ps) - (L - n) // ps for L, n in zip(lens, new)]
        keys = sum(L - (L - n) // ps * ps for L, n in zip(lens, new))
        return {"bytes": Hkv * D * (keys * e + sum(pages) * 4) + 4 * sum(pages), "flops": 2 * keys * Hkv * D}
    Hq, T = case["q_heads"], sum(rows)
    n = [_cdiv(L, ps) for L in lens]
    table = 4 * sum(n)
    if case["op"] == "select":
        # a request with no more pages than a row may take needs no scores
        scored = [(r, x) for r, x in zip(rows, n) if x > case["top"]]
        read = sum(x * (Hkv * 2 * D * 2 + 4) + r * Hq * D * 2 for r, x in scored) + 4 * len(n)
        return {"bytes": read + T * Hkv * case["top"] * 4, "flops": sum(2 * r * Hq * x * D for r, x in scored)}
    # pages of a kv head that some row of the request attends to (rows choose apart from one another)
    pages = [x * (1 - (1 - min(1.0, case["top"] / x)) ** r) for x, r in zip(n, rows)]
    keys = sum(r * min(case["top"] * ps, L) for L, r in zip(lens, rows))
    move = sum(pages) * ps * Hkv * D * 2 * e + T * Hq * (D * 4 + 4) + T * Hkv * case["top"] * 4
    return {"bytes": move, "flops": 4 * keys * Hq * D}


# ---- the definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "bounds": _exact_bounds, "select": _exact_select,
            "attend": _exact_attend}[case["op"]](s)


def _exact_append(s):
    D, rot, half = s["dim"], s["rot"], s["rot"] // 2
    table = s["cos_sin"].double()
    one = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS) * w.double()
        y = x.clone()
        pair = 0
        for axis, n in enumerate(s["sections"]):
            at = s["positions"][axis].long()
            for i in range(pair, pair + n):
                a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, half + i)
                turn = torch.complex(table[at, i], table[at, half + i])[:, None]
                z = torch.complex(x[..., a].contiguous(), x[..., b].contiguous()) * turn
                y[..., a], y[..., b] = z.real, z.imag
            pair += n
        one.append(y)
    ps = s["page"]
    caches = []
    for cache, x, scale in ((s["k_cache"], one[1], s["scale_k"]), (s["v_cache"], s["v"].double(), s["scale_v"])):
        c = _values(cache).to(torch.float64)
        if s["kv"] == "e4m3":
            x = (x / scale).clamp(-448.0, 448.0)
        c[s["slots"] // ps, s["slots"] % ps] = x
        caches.append(c)
    return one[0], caches[0], caches[1]


def _numbers64(s, codes, scale):
    if s["kv"] == "e4m3":
        return (codes.view(E4M3).to(torch.float32) * torch.tensor(scale, device="cuda")).to(torch.bfloat16).double()
    return codes.double()


def _exact_bounds(s):
    ps = s["page"]
    out = s["bounds"].double()
    for b, L in enumerate(s["lens"]):
        begin = (L - s["rows"][b]) // ps if s["new"] else 0
        ids = s["table"][b, begin:_cdiv(L, ps)].long()
        k = _numbers64(s, s["k_cache"][ids], s["scale_k"])
        out[ids[:-1], :, 0], out[ids[:-1], :, 1] = k[:-1].min(1).values, k[:-1].max(1).values
        tail = k[-1, :L - (_cdiv(L, ps) - 1) * ps]
        out[ids[-1], :, 0], out[ids[-1], :, 1] = tail.min(0).values, tail.max(0).values
    return out


def _exact_select(s):
    ps, Hkv, top = s["page"], s["kv_heads"], s["top"]
    G = s["q_heads"] // Hkv
    out = torch.full_like(s["pages"], -1)
    for b, L in enumerate(s["lens"]):
        bounds = s["bounds"][s["table"][b, :_cdiv(L, ps)].long()].double().unbind(2)    # lo, hi: [n, Hkv, D]
        begin = int(s["qsl"][b])
        for r in range(s["rows"][b]):
            n = (L - s["rows"][b] + r) // ps + 1
            q = s["q"][begin + r].double().reshape(Hkv, G, -1)
            u = torch.stack([torch.maximum(q[:, j] * bounds[0][:n], q[:, j] * bounds[1][:n]).sum(-1) for j in range(G)])
            score = u.max(0).values.t()                           # [Hkv, n]
            if n <= top:
                out[begin + r, :, :n] = torch.arange(n, device="cuda")
                continue
            score[:, :s["first"]] = math.inf
            score[:, n - s["last"]:] = math.inf
            best = torch.argsort(-score, dim=1, stable=True)[:, :top]
            out[begin + r] = best.sort(1).values.int()
    return out


def _exact_attend(s):
    ps, Hkv, D = s["page"], s["kv_heads"], s["dim"]
    G = s["q_heads"] // Hkv
    out, lse = torch.empty_like(s["out"], dtype=torch.float64), torch.empty_like(s["lse"], dtype=torch.float64)
    for b, L in enumerate(s["lens"]):
        begin = int(s["qsl"][b])
        for r in range(s["rows"][b]):
            pos = L - s["rows"][b] + r
            for h in range(Hkv):
                pages = s["pages"][begin + r, h].long()
                pages = pages[pages >= 0]
                ids = s["table"][b].long()[pages]
                seen = (pages[:, None] * ps + torch.arange(ps, device="cuda")).flatten() <= pos
                k = _numbers64(s, s["k_cache"][ids, :, h], s["scale_k"]).reshape(-1, D)[seen]
                v = _numbers64(s, s["v_cache"][ids, :, h], s["scale_v"]).reshape(-1, D)[seen]
                x = s["q"][begin + r, h * G:(h + 1) * G].double() @ k.t() / math.sqrt(D)
                if s["cap"]:
                    x = s["cap"] * torch.tanh(x / s["cap"])
                if s["sink"] is not None:
                    x = torch.cat([x, s["sink"][h * G:(h + 1) * G, None].double()], 1)
                    v = torch.cat([v, torch.zeros(1, D, dtype=torch.float64, device="cuda")])
                out[begin + r, h * G:(h + 1) * G] = torch.softmax(x, 1) @ v
                lse[begin + r, h * G:(h + 1) * G] = torch.logsumexp(x, 1)
    return out, lse
