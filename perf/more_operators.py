"""The speculative serving step over an 8-bit paged cache, operator by operator.

A step builds the block tables and slot maps of its requests on the GPU from
their lengths, appends the new tokens' keys and values to a cache of 8-bit codes
with a scale for each page and kv head, attends over that cache (one row a
request, a few drafted ones, or chunks of a prompt), and verifies the drafted
tokens against the target's probabilities.  Each case is one of the four;
``run`` computes it with elementary torch operations, or, where ``own`` is true,
by the calls of ``paged_kv_gqa_12_gb300.binding``.
"""
import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
MOST = {"int8": 127.0, "e4m3": 448.0}


# ---- cases ---------------------------------------------------------------------

def _tables(name, batch, ctx_lo, ctx_hi, new_lo, new_hi, page, ended=0):
    return dict(name=name, op="tables", batch=batch, ctx_lo=ctx_lo, ctx_hi=ctx_hi, new_lo=new_lo, new_hi=new_hi,
                page=page, ended=ended)


def _append(name, batch, ctx_lo, ctx_hi, new_lo, new_hi, kv_heads, dim, page, code):
    return dict(name=name, op="append", batch=batch, ctx_lo=ctx_lo, ctx_hi=ctx_hi, new_lo=new_lo, new_hi=new_hi,
                kv_heads=kv_heads, dim=dim, page=page, code=code)


def _attend(name, batch, ctx_lo, ctx_hi, new_lo, new_hi, q_heads, kv_heads, dim, page, code, window=0, sinks=False,
            cap=0.0):
    return dict(name=name, op="attend", batch=batch, ctx_lo=ctx_lo, ctx_hi=ctx_hi, new_lo=new_lo, new_hi=new_hi,
                q_heads=q_heads, kv_heads=kv_heads, dim=dim, page=page, code=code, window=window, sinks=sinks, cap=cap)


def _verify(name, batch, rows_lo, rows_hi, vocab, drafts=True):
    return dict(name=name, op="verify", batch=batch, rows_lo=rows_lo, rows_hi=rows_hi, vocab=vocab, drafts=drafts)


def listed():
    return [
        # a decode step of four requests: latency alone
        _tables("tables_decode_4", 4, 60, 1000, 1, 1, 16),
        # a step that starts 40 prompts beside running requests, some of which have ended
        _tables("tables_prompts_250", 250, 0, 8191, 1, 500, 16, ended=17),
        # a decode step of 64 requests
        _append("append_decode_64_int8", 64, 63, 511, 1, 1, 8, 128, 16, "int8"),
        # a verification step: one to five new tokens a request
        _append("append_verify_250_e4m3", 250, 63, 511, 1, 5, 8, 128, 64, "e4m3"),
        # a prefill step of prompts and chunks
        _append("append_prefill_8_int8", 8, 0, 300, 700, 3395, 8, 128, 16, "int8"),
        # four short requests of a small model: latency alone
        _attend("attend_decode_4_int8", 4, 60, 1000, 1, 1, 8, 2, 64, 16, "int8"),
        # a decode step of 64 requests
        _attend("attend_decode_64_int8", 64, 512, 8191, 1, 1, 32, 8, 128, 16, "int8"),
        # one request deep in a context of 131071 tokens
        _attend("attend_one_131071_e4m3", 1, 131070, 131070, 1, 1, 32, 8, 128, 16, "e4m3"),
        # a verification step of 64 requests, with sinks
        _attend("attend_verify_64_e4m3", 64, 512, 8191, 1, 4, 32, 8, 128, 16, "e4m3", sinks=True),
        # chunks of prompts of 8 requests
        _attend("attend_chunk_8_int8", 8, 0, 8191, 200, 1000, 32, 8, 128, 16, "int8"),
        # one request's four drafts, without the drafts' probabilities (taken as certain)
        _verify("verify_one_32000", 1, 5, 5, 32000, drafts=False),
        # none to four drafts of 64 requests
        _verify("verify_64_131072", 64, 1, 5, 131072),
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
    op = rng.choice(["tables", "append", "attend", "attend", "verify"])
    hq, hkv, dim = rng.choice(_HEADS)
    page = rng.choice([16, 32, 64])
    code = rng.choice(["int8", "e4m3"])
    if op == "verify":
        c = _verify("", _log_uniform(rng, 1, 64), 1, rng.randint(1, 8), _log_uniform(rng, 1000, 131072),
                    drafts=rng.random() < 0.6)
        c["rows_lo"] = rng.randint(1, c["rows_hi"])
    else:
        batch = _log_uniform(rng, 1, 250 if op != "attend" else 64)
        new = rng.choice([1, rng.randint(2, 6), _log_uniform(rng, 7, 1000)])
        lo = rng.randint(1, new)
        if op == "tables":
            hi = _log_uniform(rng, 10, 8191)
            c = _tables("", batch, int(hi * rng.random()), hi, lo, new, page, ended=rng.randint(0, batch // 4))
        elif op == "append":
            hi = _log_uniform(rng, 5, 511)
            c = _append("", batch, int(hi * rng.random()), hi, lo, new, hkv, dim, page, code)
        else:
            hi = _log_uniform(rng, 20, min(131070, 300000 // batch))
            c = _attend("", batch, int(hi * rng.random()), hi, lo, new, hq, hkv, dim, page, code,
                        window=rng.choice([0, 0, 0, _log_uniform(rng, 16, 2000)]), sinks=rng.random() < 0.3,
                        cap=rng.choice([0.0, 0.0, 30.0]))
    del c["name"]
    return c


# ---- inputs --------------------------------------------------------------------

def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]: the same for every seed, so that the work of a case is known."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _cdiv(a, b):
    return -(-a // b)


def _ctx_new(case):
    """(tokens in the cache, new tokens) of each request: long contexts go with few new tokens and with many alike."""
    B = case["batch"]
    ctx, new = _spread(case["ctx_lo"], case["ctx_hi"], B), _spread(case["new_lo"], case["new_hi"], B)
    if case["op"] == "tables":
        # most requests bring one token, every sixth a prompt; the ended ones lie among them
        new = [n if i % 6 == 0 else min(n, 1 + i % 2) for i, n in enumerate(new)]
        for i in range(case["ended"]):
            new[(i * B) // case["ended"]] = -1
        return list(zip(ctx, new))
    return [(c, new[(i * 7 + 3) % B]) for i, c in enumerate(ctx)]


def _rows(case):
    """Rows of each request of a verification: its drafts and one."""
    return _spread(case["rows_lo"], case["rows_hi"], case["batch"])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)
    s = dict(case)
    return {"tables": _prepare_tables, "append": _prepare_append, "attend": _prepare_attend,
            "verify": _prepare_verify}[case["op"]](s, g)


def _order(items, g):
    return [items[i] for i in torch.randperm(len(items), generator=g, device="cuda").tolist()]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_tables(s, g):
    B, ps = s["batch"], s["page"]
    # (some requests hold a page for later)
    some = _order([(c, n, _cdiv(c, ps) + (i % 3 == 1)) for i, (c, n) in enumerate(_ctx_new(s))], g)
    ctx, new, held = ([x[i] for x in some] for i in range(3))
    width = max(max(held), max(_cdiv(c + max(n, 0), ps) for c, n in zip(ctx, new))) + 2
    need = sum(max(0, _cdiv(c + n, ps) - h) for c, n, h in zip(ctx, new, held) if n >= 0)
    pool = sum(held) + need + 50
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = perm[at:at + n]
        at += n
    s["free_pages"] = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
    s["free_pages"][:pool - at] = perm[at:]
    s["pool"], s["table"] = pool, table
    s["ctx"], s["new"], s["held"], s["free"] = _i32(ctx), _i32(new), _i32(held), _i32([pool - at])
    tokens = sum(max(n, 0) for n in new)
    s["tokens"] = tokens + 7                    # capacity: a few padded tokens behind the last
    for name, n, dtype in (("seq", B, torch.int32), ("qsl", B + 1, torch.int32), ("slots", s["tokens"], torch.int64),
                           ("pos", s["tokens"], torch.int32), ("held_out", B, torch.int32),
                           ("free_out", 1, torch.int32)):
        s[name] = torch.zeros(n, dtype=dtype, device="cuda")
    return s


def _paged(s, g):
    """Requests in a seeded order over a shuffled pool."""
    ps = s["page"]
    pairs = _order(_ctx_new(s), g)
    s["pairs"] = pairs
    lens = [c + n for c, n in pairs]
    n_pages = [_cdiv(L, ps) for L in lens]
    pool = sum(n_pages) + 8
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(s["batch"], max(n_pages), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(n_pages):
        table[b, :n] = perm[at:at + n]
        at += n
    qsl = [0]
    for _, n in pairs:
        qsl.append(qsl[-1] + n)
    s["lens"], s["starts"], s["pool"], s["table"] = lens, qsl, pool, table
    s["seq_lens"], s["qsl"], s["total"] = _i32(lens), _i32(qsl), qsl[-1]
    s["one"] = s["new_hi"] == 1                 # a decode step: one row a request


def _codes(shape, code, g):
    """Codes as a cache holds them after blocks were scaled to their largest value."""
    out = torch.empty(shape, dtype=torch.int8 if code == "int8" else torch.uint8, device="cuda")
    for part in out.split(2048):
        x = torch.randn(part.shape, generator=g, device="cuda") * (MOST[code] / 3.5)
        x = x.clamp(-MOST[code], MOST[code])
        part.copy_(x.round().to(torch.int8) if code == "int8" else x.to(E4M3).view(torch.uint8))
    return out


def _scales(s, g, size):
    """Scales of pages whose largest values differ by a factor of four."""
    u = torch.rand(s["pool"], s["kv_heads"], generator=g, device="cuda")
    return size * 3.5 / MOST[s["code"]] * 2.0 ** (2 * u - 1)


def _prepare_append(s, g):
    _paged(s, g)
    Hkv, D, ps = s["kv_heads"], s["dim"], s["page"]
    # k and v are parts of one projection's output
    kv = torch.randn(s["total"], 2 * Hkv, D, generator=g, device="cuda").bfloat16()
    s["k"], s["v"] = kv[:, :Hkv], kv[:, Hkv:]
    s["k_cache"], s["v_cache"] = (_codes((s["pool"], ps, Hkv, D), s["code"], g) for _ in range(2))
    s["k_scales"], s["v_scales"] = _scales(s, g, 1.0), _scales(s, g, 1.0)
    s["most"] = max(_cdiv(L, ps) - (L - n) // ps for L, (_, n) in zip(s["lens"], s["pairs"]))
    return s


def _prepare_attend(s, g):
    _paged(s, g)
    Hq, Hkv, D, ps, T = s["q_heads"], s["kv_heads"], s["dim"], s["page"], s["total"]
    s["q"] = torch.randn(T, Hq, D, generator=g, device="cuda").bfloat16()
    s["k_cache"], s["v_cache"] = (_codes((s["pool"], ps, Hkv, D), s["code"], g) for _ in range(2))
    s["k_scales"], s["v_scales"] = _scales(s, g, 1.0), _scales(s, g, 1.0)
    s["sink"] = torch.randn(Hq, generator=g, device="cuda") if s["sinks"] else None
    s["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(T, Hq, dtype=torch.float32, device="cuda")
    if own:
        from paged_kv_gqa_12_gb300 import binding as pb
        s["plan"] = pb.block_plan(num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=ps,
                                  code=pb.CODE_INT8 if s["code"] == "int8" else pb.CODE_E4M3, max_batch=s["batch"],
                                  max_pages_per_seq=s["table"].shape[1], max_total_q=T, max_new=s["new_hi"],
                                  window=s["window"], has_sinks=bool(s["sinks"]), soft_cap=s["cap"],
                                  host_seq_lens=s["lens"])
        s["scratch"] = pb.alloc_scratch(s["plan"])
    return s


def _prepare_verify(s, g):
    B, V = s["batch"], s["vocab"]
    rows = _order(_rows(s), g)
    qsl = [0]
    for n in rows:
        qsl.append(qsl[-1] + n)
    T = qsl[-1]
    s["qsl"], s["starts"], s["total"], s["width"] = _i32(qsl), qsl, T, s["rows_hi"] + 1
    logits = 3.0 * torch.randn(T, V, generator=g, device="cuda")
    s["p"] = torch.softmax(logits, -1)
    # the drafting model's distribution is near the target's
    draft = torch.softmax(logits + 1.2 * torch.randn(T, V, generator=g, device="cuda"), -1)
    race = torch.empty(T, V, device="cuda").exponential_(generator=g)
    drawn = (draft / race).argmax(-1).to(torch.int32)             # a draw from each row's draft distribution
    s["drafts_p"] = draft if s["drafts"] else None
    s["tokens"] = torch.cat([drawn.new_zeros(1), drawn[:-1]])     # row r's draft is the token that follows it
    s["u"] = torch.rand(T, generator=g, device="cuda")
    s["w"] = torch.rand(B, generator=g, device="cuda")
    s["out"] = torch.empty(B, s["width"], dtype=torch.int32, device="cuda")
    s["num"] = torch.empty(B, dtype=torch.int32, device="cuda")
    return s


# ---- one pass ------------------------------------------------------------------

def run(s):
    return {"tables": _run_tables, "append": _run_append, "attend": _run_attend, "verify": _run_verify}[s["op"]](s)


def _run_tables(s):
    outs = (s["table"], s["free_pages"], s["free_out"], s["held_out"], s["seq"], s["qsl"], s["slots"], s["pos"])
    ps, pool = s["page"], s["pool"]
    if own:
        from paged_kv_gqa_12_gb300 import binding as pb
        pb.step_tables(s["ctx"], s["new"], s["held"], s["free_pages"], s["free"], s["table"], page_size=ps,
                       num_pages=pool, seq_lens=s["seq"], query_start_loc=s["qsl"], slots=s["slots"],
                       positions=s["pos"], page_counts_out=s["held_out"], free_count_out=s["free_out"])
        return outs
    B, W = s["table"].shape
    ctx, new, held = s["ctx"].long(), s["new"].long(), s["held"].long()
    ended = new < 0
    n = new.clamp(min=0)
    seq = torch.where(ended, 0, ctx + n)
    col = torch.arange(W, device="cuda")
    # the stack of free pages, with those of the ended requests on top
    gone = s["table"][ended[:, None] & (col < held[:, None])]
    stack = torch.cat([s["free_pages"][:int(s["free"])], gone])
    fresh = ~ended[:, None] & (col >= held[:, None]) & (col < ((seq + ps - 1) // ps)[:, None])
    need = int(fresh.sum())
    s["table"][fresh] = stack.flip(0)[:need]
    left = stack[:stack.shape[0] - need]
    s["free_pages"][:left.shape[0]] = left
    s["free_out"].fill_(left.shape[0])
    s["held_out"].copy_(torch.where(ended, 0, torch.maximum(held, (seq + ps - 1) // ps)))
    s["seq"].copy_(seq)
    s["qsl"].copy_(torch.nn.functional.pad(n.cumsum(0), (1, 0)))
    row = torch.arange(s["tokens"], device="cuda")
    req = torch.searchsorted(s["qsl"][1:].long(), row, right=True)
    there, req = req < B, req.clamp(max=B - 1)
    pos = ctx[req] + row - s["qsl"].long()[req]
    slot = s["table"][req, (pos // ps).clamp(max=W - 1)].long() * ps + pos % ps
    s["slots"].copy_(torch.where(there, slot, -1))
    s["pos"].copy_(torch.where(there, pos, 0))
    return outs


def _to_code(s, x):
    """The code next to x (64-bit), ties to even, and the value it stands for."""
    if s["code"] == "int8":
        q = x.round().clamp(-127.0, 127.0)
        return q.to(torch.int8)
    x = x.clamp(-448.0, 448.0)
    # steps of e4m3: 2^-9 below 2^-6, then an eighth of the power of two below x
    step = 2.0 ** (torch.frexp(x.abs().clamp(min=2.0 ** -6))[1].double() - 4)
    return ((x / step).round() * step).float().to(E4M3).view(torch.uint8)


def _values(s, codes):
    return codes.double() if s["code"] == "int8" else codes.view(E4M3).to(torch.float32).double()


def _caches(s):
    """Caches as the numbers their codes are, and the scales."""
    kc, vc = s["k_cache"], s["v_cache"]
    if s["code"] == "e4m3":
        kc, vc = kc.view(E4M3), vc.view(E4M3)
    return kc, vc, s["k_scales"], s["v_scales"]


def _run_append(s):
    if own:
        from paged_kv_gqa_12_gb300 import binding as pb
        pb.append_blocks(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"],
                         s["seq_lens"], query_start_loc=None if s["one"] else s["qsl"])
        return _caches(s)
    ps, T = s["page"], s["total"]
    L, qsl = s["seq_lens"].long(), s["qsl"].long()
    ctx = L - (qsl[1:] - qsl[:-1])
    i = (ctx // ps)[:, None] + torch.arange(s["most"], device="cuda")       # [B, most]: the pages that change
    there = i * ps < L[:, None]
    req = torch.arange(s["batch"], device="cuda")[:, None].expand_as(i)[there]
    i = i[there]
    ids = s["table"].long()[req, i]
    pos = i[:, None] * ps + torch.arange(ps, device="cuda")                  # [pages, ps]
    old, new = pos < ctx[req][:, None], (pos >= ctx[req][:, None]) & (pos < L[req][:, None])
    row = (qsl[req][:, None] + pos - ctx[req][:, None]).clamp(0, T - 1)
    for x, cache, scales in ((s["k"], s["k_cache"], s["k_scales"]), (s["v"], s["v_cache"], s["v_scales"])):
        x = x[row].float()                                                   # [pages, ps, Hkv, D]
        most = x.abs().masked_fill(~new[..., None, None], 0.0).amax((1, 3))
        was = torch.where(old.any(1)[:, None], scales[ids], 0.0)
        scale = torch.maximum(was, (most.double() / MOST[s["code"]]).float())
        safe = torch.where(scale > 0, scale, 1.0).double()[:, None, :, None]
        there_codes = cache[ids]
        grown = (scale > was)[:, None, :, None] & old[..., None, None]
        again = _to_code(s, _values(s, there_codes) * was.double()[:, None, :, None] / safe)
        codes = torch.where(grown, again, there_codes)
        codes = torch.where(new[..., None, None], _to_code(s, x.double() / safe), codes)
        cache[ids] = codes
        scales[ids] = scale
    return _caches(s)


def _run_attend(s):
    if own:
        from paged_kv_gqa_12_gb300 import binding as pb
        pb.block_attend(s["plan"], s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"],
                        s["seq_lens"], query_start_loc=None if s["one"] else s["qsl"], scale=s["dim"] ** -0.5,
                        out=s["out"], lse=s["lse"], sinks=s["sink"], scratch=s["scratch"])
        return s["out"], s["lse"]
    Hkv, D, ps = s["kv_heads"], s["dim"], s["page"]
    for b, (ctx, n) in enumerate(s["pairs"]):
        L, begin = ctx + n, s["starts"][b]
        first = max(0, (ctx - s["window"] + 1) // ps) if s["window"] else 0
        ids = s["table"][b, first:_cdiv(L, ps)].long()
        kv = []
        for cache, scales in ((s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"])):
            x = cache[ids].float() if s["code"] == "int8" else cache[ids].view(E4M3).float()
            x = (x * scales[ids][:, None, :, None]).reshape(-1, Hkv, D)[:L - first * ps]
            kv.append(x.transpose(0, 1))                                     # [Hkv, keys, D]
        q = s["q"][begin:begin + n].float().reshape(n, Hkv, -1, D).permute(1, 2, 0, 3)   # [Hkv, G, n, D]
        x = (q @ kv[0].transpose(-1, -2)[:, None]) * D ** -0.5
        if s["cap"]:
            x = s["cap"] * torch.tanh(x / s["cap"])
        at = first * ps + torch.arange(kv[0].shape[1], device="cuda")
        pos = ctx + torch.arange(n, device="cuda")[:, None]
        seen = at <= pos
        if s["window"]:
            seen = seen & (pos - at < s["window"])
        x.masked_fill_(~seen, -math.inf)
        top = x.amax(-1, keepdim=True)
        if s["sink"] is not None:
            sink = s["sink"].reshape(Hkv, -1, 1, 1)
            top = torch.maximum(top, sink)
        e = torch.exp(x - top)
        z = e.sum(-1, keepdim=True)
        if s["sink"] is not None:
            z = z + torch.exp(sink - top)
        s["out"][begin:begin + n] = ((e @ kv[1][:, None]) / z).permute(2, 0, 1, 3).reshape(n, -1, D)
        s["lse"][begin:begin + n] = (top + torch.log(z)).permute(2, 0, 1, 3).reshape(n, -1)
    return s["out"], s["lse"]


def _run_verify(s):
    if own:
        from paged_kv_gqa_12_gb300 import binding as pb
        pb.verify_tokens(s["tokens"], s["p"], s["qsl"], s["u"], s["w"], s["out"], s["num"], draft_probs=s["drafts_p"])
        return s["out"], s["num"]
    T, W = s["total"], s["width"]
    qsl = s["qsl"].long()
    n = qsl[1:] - qsl[:-1]
    # row r proposes the token of row r + 1
    draft = torch.cat([s["tokens"][1:], s["tokens"][:1]]).long()
    row = torch.arange(T, device="cuda")
    px = s["p"][row, draft].double()
    qx = s["drafts_p"][row, draft].double() if s["drafts"] else torch.ones_like(px)
    fine = s["u"].double() * qx < px
    col = torch.arange(W, device="cuda")
    at = (qsl[:-1, None] + col).clamp(max=T - 1)
    kept = (fine[at] & (col < n[:, None] - 1)).long().cumprod(1).sum(1)
    last = qsl[:-1] + kept
    # sums and the order of two of them next to a border need 64 bits
    left = s["p"][last].double()
    rejected = (kept < n - 1)[:, None]
    if s["drafts"]:
        less = left - s["drafts_p"][last].double()
    else:
        less = left.clone()
        less[torch.arange(s["batch"], device="cuda"), draft[last]] -= 1.0
    left = torch.where(rejected, less.clamp(min=0), left)
    run_sum = left.cumsum(1)
    drawn = (run_sum <= s["w"].double()[:, None] * run_sum[:, -1:]).sum(1)
    token = torch.where(col < kept[:, None], draft[at], -1)
    s["out"].copy_(torch.where(col == kept[:, None], drawn[:, None], token))
    s["num"].copy_(kept + 1)
    return s["out"], s["num"]


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    if case["op"] == "verify":
        rows, V = sum(_rows(case)), case["vocab"]
        sides = 2 if case["drafts"] else 1
        tests = (rows - case["batch"]) * (8 + 4 * sides)
        return {"bytes": case["batch"] * (V * 4 * sides + 4 * (case["rows_hi"] + 3)) + tests,
                "flops": case["batch"] * V * (sides + 1)}
    ps, pairs = case["page"], _ctx_new(case)
    if case["op"] == "tables":
        tokens = sum(max(n, 0) for _, n in pairs)
        # ids of the pages that tokens lie in, and those that are handed out or come back
        pages = sum(_cdiv(c + n, ps) - c // ps if n >= 0 else _cdiv(c, ps) for c, n in pairs)
        return {"bytes": 12 * tokens + 8 * pages + 24 * case["batch"] + 8, "flops": 4 * tokens + 8 * case["batch"]}
    Hkv, D, T = case["kv_heads"], case["dim"], sum(n for _, n in pairs)
    if case["op"] == "append":
        pages = sum(_cdiv(c + n, ps) - c // ps for c, n in pairs)
        return {"bytes": 2 * Hkv * (T * D * 3 + pages * 4) + 4 * pages + 8 * case["batch"], "flops": 2 * Hkv * T * D * 3}
    Hq, w = case["q_heads"], case["window"]
    read = [c + n - (max(0, c - w + 1) if w else 0) for c, n in pairs]       # keys that some row sees
    seen = sum(sum(min(c + i + 1, w) if w else c + i + 1 for i in range(n)) for c, n in pairs)
    pages = sum(_cdiv(r, ps) for r in read)
    return {"bytes": sum(read) * Hkv * D * 2 + pages * (Hkv * 8 + 4) + T * Hq * (D * 4 + 4), "flops": 4 * seen * Hq * D}


# ---- the definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "append": _exact_append, "attend": _exact_attend,
            "verify": _exact_verify}[case["op"]](s)


def _exact_tables(s):
    """Request by request, as an allocator on the host does it."""
    ps = s["page"]
    table, pages = s["table"].cpu(), s["free_pages"].cpu()
    ctx, new, held = s["ctx"].tolist(), s["new"].tolist(), s["held"].tolist()
    stack = pages[:int(s["free"])].tolist()
    for b, n in enumerate(new):
        if n < 0:
            stack += table[b, :held[b]].tolist()
    seq, qsl, slots, pos = [], [0], [], []
    for b, n in enumerate(new):
        if n < 0:
            held[b] = 0
            seq.append(0)
            qsl.append(qsl[-1])
            continue
        seq.append(ctx[b] + n)
        qsl.append(qsl[-1] + n)
        while held[b] * ps < seq[b]:
            table[b, held[b]] = stack.pop()
            held[b] += 1
        for p in range(ctx[b], seq[b]):
            slots.append(int(table[b, p // ps]) * ps + p % ps)
            pos.append(p)
    pages[:len(stack)] = torch.tensor(stack, dtype=torch.int32)
    more = s["tokens"] - len(slots)
    one = dict(dtype=torch.int32)
    outs = (table, pages, torch.tensor([len(stack)], **one), torch.tensor(held, **one), torch.tensor(seq, **one),
            torch.tensor(qsl, **one), torch.tensor(slots + [-1] * more), torch.tensor(pos + [0] * more, **one))
    return tuple(x.cuda() for x in outs)


def _grid(s):
    """The numbers that codes can be, ascending."""
    if s["code"] == "int8":
        return torch.arange(-127, 128, device="cuda").double()
    x = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8).view(E4M3).to(torch.float32).double()
    return x[x.isfinite()].unique()


def _nearest(s, grid, x):
    """The number of the grid next to x; between two, the one whose code is even."""
    k = torch.searchsorted(grid, x.clamp(grid[0], grid[-1]).contiguous()).clamp(1, grid.numel() - 1)
    lo, hi = grid[k - 1], grid[k]
    # (of two neighbours one is an even whole number, or an even multiple of their step)
    low_even = torch.remainder(lo / (hi - lo), 2) == 0
    up = (x - lo > hi - x) | ((x - lo == hi - x) & ~low_even)
    return torch.where(up, hi, lo)


def _exact_append(s):
    ps, most = s["page"], MOST[s["code"]]
    grid = _grid(s)
    outs = []
    for x, cache, scales in ((s["k"], s["k_cache"], s["k_scales"]), (s["v"], s["v_cache"], s["v_scales"])):
        values, scales, x = _values(s, cache), scales.clone(), x.double()
        for b, (ctx, n) in enumerate(s["pairs"]):
            for i in range(ctx // ps, _cdiv(ctx + n, ps)):
                page = int(s["table"][b, i])
                kept, end = max(0, ctx - i * ps), min(ps, ctx + n - i * ps)
                rows = x[s["starts"][b] + i * ps + kept - ctx:s["starts"][b] + i * ps + end - ctx]
                scale = (rows.abs().amax((0, 2)) / most).float()
                if kept:
                    was = scales[page].clone()
                    scale = torch.maximum(scale, was)
                    for h in (scale > was).nonzero().flatten().tolist():
                        values[page, :kept, h] = _nearest(s, grid, values[page, :kept, h] * was[h].double()
                                                          / scale[h].double())
                scales[page] = scale
                values[page, kept:end] = _nearest(s, grid, rows / scale.double()[:, None])
        outs.append((values, scales))
    codes = [v.to(torch.int8) if s["code"] == "int8" else v for v, _ in outs]
    return codes[0], codes[1], outs[0][1].double(), outs[1][1].double()


def _exact_attend(s):
    ps, Hkv, D, w = s["page"], s["kv_heads"], s["dim"], s["window"]
    G = s["q_heads"] // Hkv
    out, lse = torch.empty_like(s["out"], dtype=torch.float64), torch.empty_like(s["lse"], dtype=torch.float64)
    for b, (ctx, n) in enumerate(s["pairs"]):
        begin, ids = s["starts"][b], s["table"][b, :_cdiv(ctx + n, ps)].long()
        for h in range(Hkv):
            k = (_values(s, s["k_cache"][ids, :, h].contiguous()) * s["k_scales"][ids, h].double()[:, None, None]).reshape(-1, D)
            v = (_values(s, s["v_cache"][ids, :, h].contiguous()) * s["v_scales"][ids, h].double()[:, None, None]).reshape(-1, D)
            for r0 in range(0, n, 128):
                r1 = min(n, r0 + 128)
                lo, hi = max(0, ctx + r0 - w + 1) if w else 0, ctx + r1
                q = s["q"][begin + r0:begin + r1, h * G:(h + 1) * G].double()
                x = torch.einsum("rgd,kd->rgk", q, k[lo:hi]) / math.sqrt(D)
                if s["cap"]:
                    x = s["cap"] * torch.tanh(x / s["cap"])
                pos = torch.arange(ctx + r0, ctx + r1, device="cuda")[:, None, None]
                at = torch.arange(lo, hi, device="cuda")
                away = (at > pos) | ((at <= pos - w) if w else (at < 0))
                x = x.masked_fill(away, -math.inf)
                total = torch.logsumexp(x, -1)
                if s["sink"] is not None:
                    total = torch.logaddexp(total, s["sink"][h * G:(h + 1) * G].double())
                out[begin + r0:begin + r1, h * G:(h + 1) * G] = torch.exp(x - total[..., None]) @ v[lo:hi]
                lse[begin + r0:begin + r1, h * G:(h + 1) * G] = total
    return out, lse


def _exact_verify(s):
    """Request by request on the host."""
    tokens, u, w = s["tokens"].cpu().numpy(), s["u"].cpu().double().numpy(), s["w"].cpu().double().numpy()
    out, num = np.full((s["batch"], s["width"]), -1, np.int32), np.zeros(s["batch"], np.int32)
    for b in range(s["batch"]):
        begin, n = s["starts"][b], s["starts"][b + 1] - s["starts"][b]
        for i in range(n):
            r = begin + i
            p = s["p"][r].cpu().double().numpy()
            left = p
            if i < n - 1:
                x = int(tokens[r + 1])
                q = s["drafts_p"][r].cpu().double().numpy() if s["drafts"] else (np.arange(p.size) == x).astype(np.float64)
                if u[r] * q[x] < p[x]:
                    out[b, i] = x
                    continue
                left = np.maximum(p - q, 0.0)
            c = np.cumsum(left)
            out[b, i], num[b] = np.searchsorted(c, w[b] * c[-1], side="right"), i + 1
            break
    return torch.from_numpy(out).cuda(), torch.from_numpy(num).cuda()
