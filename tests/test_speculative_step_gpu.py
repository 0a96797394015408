"""The serving step as a server runs it: tables, append, attention and verification, step after
step on one stream, with requests that come and end, against the same loop in 64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from paged_kv_gqa_12_gb300 import binding as pb  # noqa: E402
from tests import block_refs as ref  # noqa: E402

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

_k = dict(dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_steps(kind):
    B, ps, pool, W, V = 6, 16, 60, 12, 300
    Hq, Hkv, D, most = 8, 2, 64, 4
    g = torch.Generator().manual_seed(5)
    code = pb.CODE_INT8 if kind == "int8" else pb.CODE_E4M3
    ctx, held = torch.zeros(B, **_k), torch.zeros(B, **_k)
    free, count = torch.randperm(pool, generator=g).to(torch.int32).cuda(), torch.tensor([pool], **_k)
    table = torch.zeros(B, W, **_k)
    cap = 200
    seq, qsl = torch.zeros(B, **_k), torch.zeros(B + 1, **_k)
    slots, pos = torch.zeros(cap, dtype=torch.int64, device="cuda"), torch.zeros(cap, **_k)
    dt = torch.int8 if kind == "int8" else torch.uint8
    kc, vc = torch.zeros(pool, ps, Hkv, D, dtype=dt, device="cuda"), torch.zeros(pool, ps, Hkv, D, dtype=dt, device="cuda")
    ks, vs = torch.zeros(pool, Hkv, device="cuda"), torch.zeros(pool, Hkv, device="cuda")
    plans = {n: pb.block_plan(num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=ps, code=code, max_batch=B,
                              max_pages_per_seq=W, max_total_q=cap, max_new=n) for n in (most, 60)}
    scratch = {n: pb.alloc_scratch(p) for n, p in plans.items()}
    out_tokens, num = torch.zeros(B, 60, **_k), torch.zeros(B, **_k)
    # the same state on the host, in 64 bits where numbers are computed
    h_ctx, h_held, h_count = [0] * B, [0] * B, pool
    h_free, h_table = free.cpu(), table.cpu()
    h_cache = {"k": (kc.cpu(), ks.cpu()), "v": (vc.cpu(), vs.cpu())}
    wait = [0] * B
    for step in range(9):
        new = []
        for b in range(B):
            if step == 0 or wait[b] == 1:
                new.append([7, 40, 16, 1, 33, 20][b])            # a prompt
                wait[b] = 0
            elif h_ctx[b] > 90 or (step == 4 and b == 1):
                new.append(-1)                                   # ends; comes back with a prompt
                wait[b] = 1
            else:
                new.append(1 + (b + step) % most)                # the last token and its drafts
        chunk = max(new) > most
        n_max = 60 if chunk else most
        new_t = torch.tensor(new, **_k)
        pb.step_tables(ctx, new_t, held, free, count, table, page_size=ps, num_pages=pool, seq_lens=seq,
                       query_start_loc=qsl, slots=slots, positions=pos, scratch=scratch[n_max])
        h_table, h_free, h_count, h_held, h_seq, h_qsl, h_slots, h_pos = ref.tables(
            h_ctx, new, h_held, h_free, h_count, h_table, ps, cap)
        T = h_qsl[-1]
        kv = torch.randn(T, 2 * Hkv, D, generator=g).bfloat16()
        q = torch.randn(T, Hq, D, generator=g).bfloat16()
        kvd, qd = kv.cuda(), q.cuda()
        pb.append_blocks(kvd[:, :Hkv], kvd[:, Hkv:], kc, vc, ks, vs, table, seq, query_start_loc=qsl,
                         scratch=scratch[n_max])
        out, lse = torch.empty_like(qd), torch.empty(T, Hq, device="cuda")
        pb.block_attend(plans[n_max], qd, kc, vc, ks, vs, table, seq, query_start_loc=qsl, scale=D ** -0.5, out=out,
                        lse=lse, scratch=scratch[n_max])
        p = torch.softmax(2 * torch.randn(T, V, generator=g), -1)
        d = torch.softmax(torch.log(p) + 0.5 * torch.randn(T, V, generator=g), -1)
        drawn = torch.multinomial(d, 1, generator=g).flatten().to(torch.int32)
        tokens = torch.cat([drawn.new_zeros(1), drawn[:-1]])
        u, w = torch.rand(T, generator=g), torch.rand(B, generator=g)
        pb.verify_tokens(tokens.cuda(), p.cuda(), qsl, u.cuda(), w.cuda(), out_tokens, num, draft_probs=d.cuda(),
                         scratch=scratch[n_max])
        # a request that brings a prompt keeps all of it; the others what was accepted, and one
        prompt = torch.tensor([n > most for n in new], device="cuda")
        ctx = torch.where(prompt, seq, torch.where(new_t < 0, 0, ctx + num))

        assert pb.check(scratch[n_max]) == 0
        assert torch.equal(table.cpu(), h_table) and held.tolist() == h_held and int(count) == h_count
        assert seq.tolist() == h_seq and slots.tolist() == h_slots and pos.tolist() == h_pos
        for x, rows, (cache, sc) in (("k", kv[:, :Hkv], (kc, ks)), ("v", kv[:, Hkv:], (vc, vs))):
            values, want = ref.append(kind, rows, h_cache[x][0], h_cache[x][1], h_table, h_seq, h_qsl, ps)
            assert torch.equal(ref.values(cache.cpu()), values) and torch.equal(sc.cpu(), want)
            h_cache[x] = (cache.cpu(), sc.cpu())
        o, l, to, tl = ref.attend(q, h_cache["k"][0], h_cache["v"][0], h_cache["k"][1], h_cache["v"][1], h_table, h_seq,
                                  h_qsl, D ** -0.5)
        assert ((out.cpu().double() - o).abs() <= to).all() and ((lse.cpu().double() - l).abs() <= tl).all()
        ho, hn = ref.verify(tokens, p, d, h_qsl, u, w, 60)
        assert torch.equal(out_tokens.cpu(), ho) and torch.equal(num.cpu(), hn)
        h_ctx = [L if n > most else 0 if n < 0 else c + int(k) for c, L, n, k in zip(h_ctx, h_seq, new, hn)]
        assert ctx.tolist() == h_ctx
    assert math.isfinite(float(lse.sum()))
