"""pa_sparse_attend against the definition in 64 bits, and the whole step (append
with rotation, key bounds, selection, attention) as it is used."""
import dataclasses

import numpy as np
import pytest
import torch

from paged_kv_gqa_12_gb300 import workloads as wl
from tests import gpu_helpers as gh
from tests import long_refs as lr

pytestmark = pytest.mark.gpu
MARK = 55.0


@pytest.fixture(scope="module")
def pb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_12_gb300 import binding
    binding.load()
    return binding


def make(lens, Hq, Hkv, D, ps, *, top, rows=None, kv="bf16", seed=0, sinks=False, cap=0.0, extra_rows=0, fill=1.0,
         shuffle=False, **kw):
    """A poisoned paged problem and a seeded choice of pages for each row: about `fill` of top, the row's own page
    among them, shuffled or ascending, then -1."""
    scales = dict(k_scale=0.05, v_scale=0.04) if kv == "fp8_e4m3" else {}
    mode = "decode" if rows is None else "extend"
    p = wl.build_problem(mode, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=ps, seq_lens=lens,
                         query_lens=rows, kv_dtype=kv, seed=seed, sinks=sinks, soft_cap=cap, **{**scales, **kw})
    rng = np.random.default_rng(seed + 1)
    qsl = None if rows is None else p.query_start_loc.tolist()
    T = p.num_rows + extra_rows
    q = torch.cat([gh._t(p.q), torch.ones(extra_rows, Hq, D, dtype=torch.bfloat16)])
    pages = torch.full((T, Hkv, top), -1, dtype=torch.int32)
    for row, b, pos in lr.rows_of(list(lens), qsl):
        n = pos // ps + 1 if pos >= 0 else 0
        for h in range(Hkv):
            k = min(n, max(1, int(round(top * fill * rng.uniform(0.5, 1.0)))), top)
            pick = rng.choice(n, size=k, replace=False) if k else np.zeros(0, int)
            if k and n - 1 not in pick:
                pick[0] = n - 1
            pick = rng.permutation(pick) if shuffle else np.sort(pick)
            pages[row, h, :k] = torch.from_numpy(pick.astype(np.int32))
    return p, dict(q=q, pages=pages, qsl=qsl, T=T, top=top)


def plan_of(pb, p, d, num_splits=0, max_total_q=None):
    return pb.sparse_plan(num_q_heads=p.num_q_heads, num_kv_heads=p.num_kv_heads, head_dim=p.head_dim,
                          page_size=p.page_size, kv_dtype=pb.KV_FP8_E4M3 if p.kv_dtype == "fp8_e4m3" else pb.KV_BF16,
                          max_batch=p.batch, max_pages_per_seq=p.block_table.shape[1],
                          max_total_q=max_total_q or d["T"], top_pages=d["top"], first_pages=0, last_pages=1,
                          has_sinks=p.sinks is not None, soft_cap=p.soft_cap, num_splits=num_splits)


def run(pb, p, d, num_splits=0, code=0, dev=None, stream=None, plan=None, scratch=None, lse=True, q=None, out=None):
    dev = dev or gh.upload(p)
    plan = plan or plan_of(pb, p, d, num_splits)
    scratch = pb.alloc_scratch(plan) if scratch is None else scratch
    q = d["q"].cuda() if q is None else q
    out = torch.full(d["q"].shape, MARK, dtype=torch.bfloat16, device="cuda") if out is None else out
    l = torch.full(d["q"].shape[:2], MARK, device="cuda") if lse else None
    pages = d["pages"].cuda()
    torch.cuda.synchronize()
    pb.sparse_attend(plan, q, dev["k"], dev["v"], dev["bt"], dev["sl"], pages, query_start_loc=dev["qsl"],
                     scale=p.scale, out=out, lse=l, sinks=dev["sinks"], k_scale=p.k_scale, v_scale=p.v_scale,
                     k_scales=dev["k_scales"], v_scales=dev["v_scales"], scratch=scratch, stream=stream)
    assert pb.check(scratch, stream) == code
    torch.cuda.synchronize()
    return out.cpu(), None if l is None else l.cpu()


def check(p, d, got, skip=()):
    out, lse = got
    kc, vc = gh._t(np.ascontiguousarray(p.k_cache)), gh._t(np.ascontiguousarray(p.v_cache))
    want = lr.attend(d["q"], kc, vc, p.block_table, p.seq_lens.tolist(), d["pages"], page_size=p.page_size,
                     scale=p.scale, query_start_loc=d["qsl"], sinks=None if p.sinks is None else torch.from_numpy(p.sinks),
                     soft_cap=p.soft_cap, k_scale=p.k_scale, v_scale=p.v_scale, k_scales=p.k_scales, v_scales=p.v_scales)
    for row in range(d["T"]):
        if row not in want or row in skip:
            assert (out[row] == MARK).all(), row
            assert lse is None or (lse[row] == MARK).all(), row
            continue
        o, l, spread = want[row]
        err = (out[row].double() - o).abs()
        tol = lr.attend_tolerance(o, spread)
        assert (err <= tol).all(), (row, (err / tol).max())
        if lse is not None:
            assert torch.equal(torch.isneginf(l), torch.isneginf(lse[row])), row
            fin = torch.isfinite(l)
            # 2^-12 for the scores (half of what the output allows for them), and 2^-20 of the value for log2 and the fp32 lse
            assert ((lse[row].double() - l).abs()[fin] <= 2.0 ** -12 + 2.0 ** -20 * l.abs()[fin]).all(), row


SHAPES = [(8, 2, 64, 16), (32, 8, 128, 16), (16, 8, 256, 32), (24, 8, 128, 64), (8, 8, 64, 64), (40, 2, 128, 16),
          (28, 4, 256, 64), (24, 2, 64, 32)]


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,ps", SHAPES)
def test_decode(pb, kv, Hq, Hkv, D, ps):
    lens = [0, 1, ps - 1, ps, ps + 1, 3 * ps + 5, 40 * ps + 9]
    for i, (top, opts) in enumerate([(9, {}), (1, dict(sinks=True)), (40, dict(cap=30.0)),
                                     (16, dict(sinks=True, cap=20.0, shuffle=True))]):
        p, d = make(lens, Hq, Hkv, D, ps, top=top, kv=kv, seed=Hq + i, **opts)
        for splits in (0, 1, 3):
            check(p, d, run(pb, p, d, num_splits=splits))


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,ps", SHAPES)
def test_packed_rows(pb, kv, Hq, Hkv, D, ps):
    lens, rows = [6 * ps + 3, 5, 0, ps, 30 * ps + 7], [9, 5, 0, 1, 4]
    p, d = make(lens, Hq, Hkv, D, ps, top=11, rows=rows, kv=kv, seed=Hq, extra_rows=3)
    for splits in (0, 1, 2):
        check(p, d, run(pb, p, d, num_splits=splits))


@pytest.mark.parametrize("Hq,D,kv", [(128, 64, "bf16"), (96, 256, "bf16"), (65, 128, "fp8_e4m3"), (33, 256, "fp8_e4m3")])
def test_large_groups(pb, Hq, D, kv):
    p, d = make([300, 45], Hq, 1, D, 16, top=7, kv=kv, seed=Hq, sinks=True)
    check(p, d, run(pb, p, d))
    check(p, d, run(pb, p, d, num_splits=3))


def test_rows_without_pages(pb):
    for sinks in (False, True):
        p, d = make([100, 200], 8, 2, 64, 16, top=6, seed=1, sinks=sinks)
        d["pages"][0, 1] = -1
        d["pages"][1, 0, 1:] = -1
        check(p, d, run(pb, p, d))
        check(p, d, run(pb, p, d, num_splits=4))


def test_negative_entries_are_passed_over(pb):
    p, d = make([300, 400], 8, 2, 128, 16, top=10, seed=2)
    d["pages"][:, :, 4] = -1
    check(p, d, run(pb, p, d))


def test_pages_behind_the_query_add_nothing(pb):
    p, d = make([100, 37], 8, 2, 64, 16, top=8, seed=3, fill=0.3)
    got = run(pb, p, d)
    more = d["pages"].clone()
    for row in range(2):
        for h in range(2):
            n = int((more[row, h] >= 0).sum())
            more[row, h, n:] = torch.tensor([10 ** 9, 7, 50, 2 ** 31 - 1, 9, 8, 30, 31][: 8 - n], dtype=torch.int32)
    for splits in (0, 3):
        again = run(pb, p, dict(d, pages=more), num_splits=splits)
        check(p, d, again)
    check(p, d, got)


def test_every_page_equals_dense_decode(pb):
    p = wl.build_problem("decode", num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16,
                         seq_lens=[500, 33, 1, 700], seed=4)
    n = p.block_table.shape[1]
    pages = torch.full((4, 8, n), -1, dtype=torch.int32)
    for b, L in enumerate(p.seq_lens.tolist()):
        pages[b, :, :-(-L // 16)] = torch.arange(-(-L // 16), dtype=torch.int32)
    d = dict(q=gh._t(p.q), pages=pages, qsl=None, T=4, top=n)
    out, lse = run(pb, p, d)
    dense, dense_lse = gh.run(p)
    check(p, d, (out, lse))
    # both are within the same bound of the exact result
    assert np.abs(out.float().numpy() - dense).max() < 1e-2 and np.abs(lse.numpy() - dense_lse).max() < 2.0 ** -11


def test_peaked_rows(pb):
    # a few keys carry a row's weight: their bf16 rounding would not average out
    p, d = make([400, 90, 260], 8, 2, 128, 16, top=20, seed=5)
    d["q"] = (d["q"].float() * 7).bfloat16()
    out, lse = run(pb, p, d)
    kc, vc = gh._t(p.k_cache), gh._t(p.v_cache)
    want = lr.attend(d["q"], kc, vc, p.block_table, p.seq_lens.tolist(), d["pages"], page_size=16, scale=p.scale)
    for row, (o, l, spread) in want.items():
        # seven times the scores, so seven times their error
        tol = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 7 * 2.0 ** -11) * spread
        assert ((out[row].double() - o).abs() <= tol).all()


def test_infinity_and_nan_in_masked_slots_and_other_heads(pb):
    p, d = make([77, 200], 8, 2, 64, 16, top=13, seed=6)
    dev = gh.upload(p)
    clean = run(pb, p, d, dev=dev)
    page = int(p.block_table[0, 4])
    dev["k"][page, 13:] = float("inf")           # slots behind the end (77 = 4 * 16 + 13)
    dev["v"][page, 13:] = float("-inf")
    got = run(pb, p, d, dev=dev)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    dev["k"][page, 2, 1, 5] = float("nan")       # an attended key of kv head 1: its four heads turn NaN, no others
    got = run(pb, p, d, dev=dev)
    assert torch.equal(got[0][0, :4], clean[0][0, :4]) and torch.equal(got[0][1], clean[0][1])
    assert got[0][0, 4:].isnan().all()


def test_page_outside_the_pool_reads_as_zeros(pb):
    p, d = make([200, 100], 8, 2, 64, 16, top=5, seed=7)
    dev = gh.upload(p)
    page = int(d["pages"][0, 0, 0])
    dev["bt"][0, page] = p.num_pages
    got = run(pb, p, d, dev=dev, code=pb.DEVICE_PAGE_ID)
    q = dataclasses.replace(p, k_cache=p.k_cache.copy(), v_cache=p.v_cache.copy())
    q.k_cache[p.block_table[0, page]] = 0
    q.v_cache[p.block_table[0, page]] = 0
    check(q, d, got)


def test_bad_requests_are_untouched(pb):
    p, d = make([200, 100, 50], 8, 2, 64, 16, top=5, seed=8)
    dev = gh.upload(p)
    dev["sl"][1] = p.block_table.shape[1] * 16 + 1
    check(p, d, run(pb, p, d, dev=dev, code=pb.DEVICE_CAPACITY), skip=(1,))
    dev["sl"][1] = -5
    check(p, d, run(pb, p, d, dev=dev, code=pb.DEVICE_CAPACITY), skip=(1,))


def test_strides_layout_and_no_lse(pb):
    p, d = make([200, 100], 8, 2, 128, 16, top=7, seed=9, layout="interleaved")
    q = torch.zeros(2, 11, 130, dtype=torch.bfloat16, device="cuda")[:, 1:9, :128]
    q.copy_(d["q"])
    out = torch.full((2, 9, 134), MARK, dtype=torch.bfloat16, device="cuda")[:, :8, 2:130]
    got = run(pb, p, d, q=q, out=out, lse=False)
    check(p, d, got)


def test_request_scales(pb):
    p, d = make([200, 100, 31], 8, 2, 64, 32, top=4, seed=10, kv="fp8_e4m3", k_scales=[0.05, 0.02, 0.09],
                v_scales=[0.03, 0.07, 0.05])
    check(p, d, run(pb, p, d))


def test_row_counts_of_one_plan(pb):
    # one plan and scratch for calls of different row counts: the split counts differ, the counters stay clean
    p, d = make([2000, 1500, 900, 1200, 800], 8, 2, 64, 16, top=60, seed=11)
    plan = plan_of(pb, p, d, max_total_q=64)
    scratch = pb.alloc_scratch(plan)
    for n in (5, 1, 3, 5):
        lens = p.seq_lens[:n]
        q = dataclasses.replace(p, q=p.q[:n], block_table=p.block_table[:n], seq_lens=lens)
        e = dict(q=d["q"][:n], pages=d["pages"][:n].contiguous(), qsl=None, T=n, top=60)
        check(q, e, run(pb, q, e, plan=plan, scratch=scratch))
    assert not scratch[:pb.SCRATCH_HEADER_BYTES].any()


def test_many_rows(pb):
    # more (row, kv head) pairs than the header has counters: one split each
    rows = [2500]
    p, d = make([2500 + 400], 8, 8, 64, 64, top=3, rows=rows, seed=12)
    out, lse = run(pb, p, d)
    some = [0, 1, 777, 1600, 2499]
    kc, vc = gh._t(p.k_cache), gh._t(p.v_cache)
    for row in some:
        sub = lr.attend(d["q"][row:row + 1], kc, vc, p.block_table, [400 + row + 1], d["pages"][row:row + 1],
                        page_size=64, scale=p.scale)
        o, l, spread = sub[0]
        assert ((out[row].double() - o).abs() <= lr.attend_tolerance(o, spread)).all()
    assert torch.isfinite(lse).all() and (out != MARK).any(-1).all()


def test_long_list(pb):
    p, d = make([4096 * 16 + 100], 4, 1, 64, 16, top=4096, seed=13)
    check(p, d, run(pb, p, d))
    check(p, d, run(pb, p, d, num_splits=1))


def test_pool_beyond_32_bit_offsets(pb):
    Hkv, D, ps = 8, 128, 16
    pool = (1 << 31) // (ps * Hkv * D) + 64
    k = torch.zeros(pool, ps, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator().manual_seed(14)
    ids = torch.tensor([[3, pool - 1, pool - 33, pool // 2, pool - 2]], dtype=torch.int32)
    kr, vr = (torch.randn(5, ps, Hkv, D, generator=g).bfloat16() for _ in range(2))
    k[ids[0].long().cuda()], v[ids[0].long().cuda()] = kr.cuda(), vr.cuda()
    q = torch.randn(1, 16, D, generator=g).bfloat16()
    pages = torch.tensor([0, 1, 2, 4], dtype=torch.int32).expand(1, Hkv, 4).contiguous()
    plan = pb.sparse_plan(num_q_heads=16, num_kv_heads=Hkv, head_dim=D, page_size=ps, max_batch=1, max_pages_per_seq=5,
                          max_total_q=1, top_pages=4)
    scratch = pb.alloc_scratch(plan)
    out = torch.empty(1, 16, D, dtype=torch.bfloat16, device="cuda")
    L = 5 * ps - 3
    pb.sparse_attend(plan, q.cuda(), k, v, ids.cuda(), torch.tensor([L], dtype=torch.int32, device="cuda"), pages.cuda(),
                     scale=D ** -0.5, out=out, scratch=scratch)
    assert pb.check(scratch) == 0
    o, _, spread = lr.attend(q, kr, vr, torch.arange(5)[None], [L], pages, page_size=ps, scale=D ** -0.5)[0]
    assert ((out[0].cpu().double() - o).abs() <= lr.attend_tolerance(o, spread)).all()


def test_two_graphs_with_one_workspace_replayed_in_turn(pb):
    a = make([500, 300], 8, 2, 64, 16, top=9, seed=15)
    b = make([400, 900], 8, 2, 64, 16, top=9, seed=16)
    graphs = []
    scratch = max((pb.alloc_scratch(plan_of(pb, p, d)) for p, d in (a, b)), key=lambda x: x.numel())
    for p, d in (a, b):
        dev, plan = gh.upload(p), plan_of(pb, p, d)
        q, pages = d["q"].cuda(), d["pages"].cuda()
        out, lse = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 8, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pb.sparse_attend(plan, q, dev["k"], dev["v"], dev["bt"], dev["sl"], pages, scale=p.scale, out=out, lse=lse,
                             scratch=scratch)
        graphs.append((graph, out, lse, dev, q, pages))
    for _ in range(3):
        for graph, *_ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for (p, d), (_, out, lse, *_) in zip((a, b), graphs):
        check(p, d, (out.cpu(), lse.cpu()))


def test_other_stream(pb):
    p, d = make([500, 300], 8, 2, 64, 16, top=9, seed=17)
    check(p, d, run(pb, p, d, stream=torch.cuda.Stream()))


def test_two_streams_at_a_time(pb):
    # two calls in flight, each with its workspace: the results are those of one at a time
    jobs = []
    for seed in (21, 22):
        p, d = make([3000, 2000, 50, 1700], 16, 4, 128, 16, top=48, seed=seed)
        plan = pb.sparse_plan(num_q_heads=16, num_kv_heads=4, head_dim=128, page_size=16, max_batch=4,
                              max_pages_per_seq=p.block_table.shape[1], max_total_q=4, top_pages=48)
        dev = gh.upload(p)
        bounds = torch.zeros(p.num_pages, 4, 2, 128, dtype=torch.bfloat16, device="cuda")
        pb.page_bounds(dev["k"], dev["bt"], dev["sl"], bounds)
        jobs.append(dict(plan=plan, dev=dev, bounds=bounds, q=d["q"].cuda(), scratch=pb.alloc_scratch(plan),
                         stream=torch.cuda.Stream(), scale=p.scale))

    def step(j, stream):
        pages = torch.empty(4, 4, 48, dtype=torch.int32, device="cuda")
        out, lse = torch.empty_like(j["q"]), torch.empty(4, 16, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        d = j["dev"]
        for _ in range(20):
            pb.select_pages(j["plan"], j["q"], j["bounds"], d["bt"], d["sl"], pages, scratch=j["scratch"], stream=stream)
            pb.sparse_attend(j["plan"], j["q"], d["k"], d["v"], d["bt"], d["sl"], pages, scale=j["scale"], out=out,
                             lse=lse, scratch=j["scratch"], stream=stream)
        return pages, out, lse

    alone = []
    for j in jobs:
        alone.append([x.cpu() for x in step(j, None)])
    both = [step(j, j["stream"]) for j in jobs]
    torch.cuda.synchronize()
    for j, a, b in zip(jobs, alone, both):
        assert pb.check(j["scratch"]) == 0
        for x, y in zip(a, b):
            assert torch.equal(x, y.cpu())


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("chunk", [False, True])
def test_whole_step(pb, kv, chunk):
    """Append with norm and rotation, refresh the bounds, select, attend: each result against its definition on the
    arrays that the step before wrote."""
    ctx, new = [700, 0, 333, 1200], [9, 12, 1, 30] if chunk else [1, 1, 1, 1]
    Hq, Hkv, D, ps, top = 16, 4, 128, 16, 10
    L = [c + n for c, n in zip(ctx, new)]
    scales = dict(k_scale=0.05, v_scale=0.04) if kv == "fp8_e4m3" else {}
    p = wl.build_problem("extend", num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=ps, seq_lens=L,
                         query_lens=new, kv_dtype=kv, seed=18, **scales)
    T = sum(new)
    g = torch.Generator().manual_seed(19)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
    pos = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)]).to(torch.int32)
    slots = torch.tensor([int(p.block_table[b, (c + i) // ps]) * ps + (c + i) % ps
                          for b, (c, n) in enumerate(zip(ctx, new)) for i in range(n)])
    freq = 1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    angle = torch.arange(2048, dtype=torch.float64)[:, None] * freq
    cs = torch.cat([angle.cos(), angle.sin()], 1).float()
    w = (1 + 0.1 * torch.randn(D, generator=g)).bfloat16()
    dev = gh.upload(p)
    kvd = pb.KV_FP8_E4M3 if kv == "fp8_e4m3" else pb.KV_BF16
    rope = pb.rope(cs.cuda(), rot_dim=D, q_norm=w.cuda(), k_norm=w.cuda())
    plan = pb.sparse_plan(num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=ps, kv_dtype=kvd, max_batch=4,
                          max_pages_per_seq=p.block_table.shape[1], max_total_q=64, top_pages=top)
    scratch = pb.alloc_scratch(plan)
    bounds = torch.zeros(p.num_pages, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    ctx_t = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    pb.page_bounds(dev["k"], dev["bt"], ctx_t, bounds, kv_dtype=kvd, k_scale=p.k_scale, scratch=scratch)
    q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, MARK), torch.full((T, Hq), MARK, device="cuda")
    pages = torch.empty(T, Hkv, top, dtype=torch.int32, device="cuda")
    pos_d, slots_d = pos.cuda(), slots.cuda()

    def step():
        pb.append_rope_kv(rope, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pos_d, dev["k"], dev["v"], slots_d,
                          q=qkv[:, :Hq], q_out=q, kv_dtype=kvd, k_scale=p.k_scale, v_scale=p.v_scale, scratch=scratch)
        pb.page_bounds(dev["k"], dev["bt"], dev["sl"], bounds, query_start_loc=dev["qsl"], kv_dtype=kvd,
                       k_scale=p.k_scale, scratch=scratch)
        pb.select_pages(plan, q, bounds, dev["bt"], dev["sl"], pages, query_start_loc=dev["qsl"], scratch=scratch)
        pb.sparse_attend(plan, q, dev["k"], dev["v"], dev["bt"], dev["sl"], pages, query_start_loc=dev["qsl"],
                         scale=p.scale, out=out, lse=lse, k_scale=p.k_scale, v_scale=p.v_scale, scratch=scratch)

    def check_step():
        kc, vc = dev["k"].cpu(), dev["v"].cpu()
        want, m = lr.norm_rotate(qkv[:, :Hq].cpu(), w, pos[None], cs, rot=D, interleaved=False, sections=(D // 2,),
                                 eps=1e-6, offset=0.0)
        assert ((q.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * m).all()
        ref = lr.bounds_of(kc, p.block_table, L, ps, p.k_scale)
        assert all(torch.equal(bounds[i].cpu().double(), v) for i, v in ref.items())
        chosen = lr.select(q.cpu(), bounds.cpu(), torch.from_numpy(p.block_table), L, page_size=ps, num_kv_heads=Hkv,
                           top=top, first=1, last=2, query_start_loc=p.query_start_loc.tolist())
        assert all(torch.equal(pages[r].cpu(), v) for r, v in chosen.items()) and len(chosen) == T
        res = lr.attend(q.cpu(), kc, vc, p.block_table, L, pages.cpu(), page_size=ps, scale=p.scale,
                        query_start_loc=p.query_start_loc.tolist(), k_scale=p.k_scale, v_scale=p.v_scale)
        for r, (o, l, spread) in res.items():
            assert ((out[r].cpu().double() - o).abs() <= lr.attend_tolerance(o, spread)).all()
            assert ((lse[r].cpu().double() - l).abs() <= 2.0 ** -12 + 2.0 ** -20 * l.abs()).all()

    step()
    assert pb.check(scratch) == 0
    check_step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    qkv.copy_(torch.randn(qkv.shape, generator=g).bfloat16())
    out.fill_(MARK)
    graph.replay()
    assert pb.check(scratch) == 0
    check_step()
