"""pa_block_attend against the definition in 64 bits, within bounds derived from its roundings
(tests/block_refs.py, attend)."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from paged_kv_gqa_12_gb300 import binding as pb  # noqa: E402
from tests import block_refs as ref  # noqa: E402

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

KINDS = {"int8": pb.CODE_INT8, "e4m3": pb.CODE_E4M3}


def _problem(seed, kind, Hq, Hkv, D, ps, ctx, new, window=0, sinks=False, cap=0.0, spread=2.0, dirty=True):
    g = torch.Generator().manual_seed(seed)
    seq = [c + n for c, n in zip(ctx, new)]
    pages = [-(-L // ps) for L in seq]
    pool = sum(pages) + 3
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    table = torch.full((len(ctx), max(pages + [1]) + 1), pool + 5, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    qsl = [0]
    for n in new:
        qsl.append(qsl[-1] + n)
    T = qsl[-1]
    s = dict(kind=kind, Hq=Hq, Hkv=Hkv, D=D, ps=ps, ctx=ctx, new=new, seq=seq, qsl=qsl, table=table, window=window,
             cap=cap, scale=D ** -0.5, q=torch.randn(T, Hq, D, generator=g).bfloat16(),
             sinks=torch.randn(Hq, generator=g) if sinks else None)
    for x in ("k", "v"):
        c = torch.randn(pool, ps, Hkv, D, generator=g) * (ref.MOST[kind] / 3.5)
        c = c.clamp(-ref.MOST[kind], ref.MOST[kind])
        s[x + "_cache"] = c.round().to(torch.int8) if kind == "int8" else c.to(ref.E4M3).view(torch.uint8)
        s[x + "_scales"] = 3.5 / ref.MOST[kind] * spread ** (2 * torch.rand(pool, Hkv, generator=g) - 1)
        if dirty:
            # what no row attends to is garbage: slots behind the end, pages of no request, pages before the window
            used = torch.zeros(pool, dtype=torch.bool)
            for b, L in enumerate(seq):
                lo = max(0, ctx[b] - window + 1) // ps if window else 0
                for i in range(lo, pages[b]):
                    used[int(table[b, i])] = True
                if L % ps:
                    s[x + "_cache"][int(table[b, pages[b] - 1]), L % ps:] = 0x7f if kind == "e4m3" else 127
            s[x + "_cache"][~used] = 0x7f if kind == "e4m3" else 127
            s[x + "_scales"][~used] = math.nan
    return s


def _plan(s, **kw):
    a = dict(num_q_heads=s["Hq"], num_kv_heads=s["Hkv"], head_dim=s["D"], page_size=s["ps"], code=KINDS[s["kind"]],
             max_batch=len(s["seq"]), max_pages_per_seq=s["table"].shape[1], max_total_q=s["q"].shape[0],
             max_new=max(s["new"] + [1]), window=s["window"], has_sinks=s["sinks"] is not None, soft_cap=s["cap"])
    a.update(kw)
    return pb.block_plan(**a)


def _dev(s):
    d = {k: s[k].cuda() for k in ("q", "k_cache", "v_cache", "k_scales", "v_scales", "table")}
    d["seq"] = torch.tensor(s["seq"], dtype=torch.int32, device="cuda")
    d["qsl"] = torch.tensor(s["qsl"], dtype=torch.int32, device="cuda")
    d["sinks"] = None if s["sinks"] is None else s["sinks"].cuda()
    d["out"] = torch.full_like(d["q"], 7.0)
    d["lse"] = torch.full(d["q"].shape[:2], 7.0, device="cuda")
    return d


def _call(s, d, plan, scratch, decode=False):
    pb.block_attend(plan, d["q"], d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"], d["table"], d["seq"],
                    query_start_loc=None if decode else d["qsl"], scale=s["scale"], out=d["out"], lse=d["lse"],
                    sinks=d["sinks"], scratch=scratch)


def _run(s, decode=False, plan=None):
    plan = plan or _plan(s)
    d = _dev(s)
    scratch = pb.alloc_scratch(plan)
    _call(s, d, plan, scratch, decode)
    return d["out"].cpu(), d["lse"].cpu(), pb.check(scratch), plan


def _want(s, decode=False):
    return ref.attend(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"], s["seq"],
                      None if decode else s["qsl"], s["scale"], s["window"], s["sinks"], s["cap"],
                      chunked=bool(_plan(s).chunked))


def _close(got, want, what=""):
    out, lse = got[0].double(), got[1].double()
    o, l, to, tl = want
    assert out.isfinite().all(), what
    e = (out - o).abs()
    assert (e <= to).all(), (what, float((e - to).max()), float((e / to.clamp(min=1e-30)).max()))
    inf = l == -math.inf
    assert torch.equal(lse == -math.inf, inf)
    d = (lse - l).abs()[~inf]
    assert d.numel() == 0 or (d <= tl[~inf]).all(), (what, float((d - tl[~inf]).max()))


LENS = [1, 15, 16, 17, 31, 32, 33, 64, 100, 500, 1037, 0]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ps", [16, 32, 64])
def test_decode(kind, D, ps):
    for Hq, Hkv in ((8, 2), (3, 3), (24, 1)):
        s = _problem(D + ps + Hq, kind, Hq, Hkv, D, ps, [max(0, L - 1) for L in LENS], [1 if L else 0 for L in LENS])
        s["q"] = torch.randn(len(LENS), Hq, D, generator=torch.Generator().manual_seed(3)).bfloat16()
        got = _run(s, decode=True, plan=_plan(s, max_total_q=len(LENS)))
        assert got[2] == 0
        _close(got, _want(s, decode=True), (Hq, Hkv))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("opts", [dict(window=1), dict(window=40), dict(window=700, sinks=True), dict(sinks=True),
                                  dict(cap=30.0), dict(cap=5.0, window=100, sinks=True)])
@pytest.mark.parametrize("ctas", [0, 1, 3, 17])
def test_decode_options(kind, opts, ctas):
    n = len(LENS) - 1
    s = _problem(77, kind, 8, 2, 128, 16, [L - 1 for L in LENS[:-1]], [1] * n, **opts)
    got = _run(s, decode=True, plan=_plan(s, num_ctas=ctas))
    assert got[2] == 0
    _close(got, _want(s, decode=True))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (32, 8, 128), (6, 2, 128), (16, 8, 256), (20, 2, 64)])
@pytest.mark.parametrize("most", [2, 5, 12])
@pytest.mark.parametrize("opts", [dict(), dict(window=50, sinks=True, cap=20.0)])
def test_a_few_rows(kind, Hq, Hkv, D, most, opts):
    ctx = [0, 3, 15, 16, 200, 777, 40, 63, 1200]
    new = [1 + i % most for i in range(9)]
    new[4] = 0
    s = _problem(most + D, kind, Hq, Hkv, D, 16, ctx, new, **opts)
    got = _run(s)
    assert got[2] == 0 and got[3].chunked == 0
    _close(got, _want(s))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,ps", [(8, 2, 64, 16), (32, 8, 128, 16), (28, 4, 128, 64), (16, 8, 256, 32),
                                         (6, 1, 256, 16), (40, 2, 128, 32)])
@pytest.mark.parametrize("opts", [dict(), dict(window=100, sinks=True), dict(cap=20.0), dict(window=1, cap=30.0, sinks=True)])
def test_chunks(kind, Hq, Hkv, D, ps, opts):
    ctx = [0, 5, 130, 0, 400, 64]
    new = [150, 1, 77, 0, 33, 64]
    s = _problem(D + Hq, kind, Hq, Hkv, D, ps, ctx, new, **opts)
    got = _run(s)
    assert got[2] == 0 and got[3].chunked == 1
    _close(got, _want(s))


def test_chunks_in_groups_of_requests():
    # a plan whose copy holds two requests at a time
    s = _problem(5, "int8", 8, 2, 64, 16, [0, 100, 7, 300, 0], [40, 33, 20, 90, 65])
    wide = 1 << 17
    table = torch.zeros(5, wide, dtype=torch.int32)
    table[:, :s["table"].shape[1]] = s["table"]
    s["table"] = table
    plan = _plan(s)
    assert plan.chunked == 1 and 1 <= plan.group_requests <= 2
    got = _run(s, plan=plan)
    assert got[2] == 0
    _close(got, _want(s))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("many", [False, True])
def test_scales_of_any_size(kind, many):
    # pages whose scales lie 2^30 apart, zeros among them; rows whose weight sits on the small ones
    new = [40, 40] if many else [1, 3]
    s = _problem(9, kind, 8, 2, 128, 16, [200, 333], new, spread=1.0)
    g = torch.Generator().manual_seed(1)
    s["v_scales"] *= 2.0 ** torch.randint(-30, 3, s["v_scales"].shape, generator=g)
    s["v_scales"][::5] = 0.0
    s["k_scales"][::3] *= 2.0 ** -20
    s["k_scales"][1::7] = 0.0
    got = _run(s)
    assert got[2] == 0
    _close(got, _want(s))
    s["v_scales"] = torch.where(s["v_scales"] > 0, 2.0 ** -90, 0.0).float()      # next to the smallest that count
    _close(_run(s), _want(s))


@pytest.mark.parametrize("many", [False, True])
def test_a_small_page_beside_a_huge_one(many):
    # the page that takes all the weight has values 2^25 below those of a page that takes none
    new = [70] if many else [2]
    s = _problem(19, "int8", 4, 2, 64, 16, [160], new, spread=1.0)
    first = int(s["table"][0, 0])
    s["k_cache"][first] = 0
    s["v_scales"][first] *= 2.0 ** 25
    s["q"][:] = s["q"].abs() * 4                     # scores of the other pages: large, with keys of one sign
    for i in range(1, -(-s["seq"][0] // 16)):
        page = int(s["table"][0, i])
        s["k_cache"][page] = s["k_cache"][page].abs()
    got = _run(s)
    _close(got, _want(s))


def test_q_of_any_size():
    s = _problem(10, "int8", 8, 2, 128, 16, [99, 400, 30, 64], [1, 1, 1, 1])
    s["q"][0] *= 2.0 ** -120
    s["q"][1] *= 2.0 ** -20
    s["q"][1, 0, 0] = 300.0                          # one large element beside small ones
    s["q"][2] = 0
    s["q"][3] *= 2.0 ** 4
    got = _run(s, decode=True)
    _close(got, _want(s, decode=True))


def test_peaked_and_flat_weights():
    # a key that takes nearly all, then keys that all weigh the same: neither rounding is one-sided
    s = _problem(11, "int8", 8, 2, 128, 16, [3000, 3000], [1, 1], spread=1.0)
    s["q"][0] *= 12
    s["q"][1] = 0
    got = _run(s, decode=True)
    _close(got, _want(s, decode=True))


def test_rows_behind_the_last_and_requests_that_do_not_fit():
    for new, plan_new in (([2, 3, 2, 4], 4), ([70, 3, 2, 4], 70)):
        s = _problem(12, "int8", 8, 2, 64, 16, [30, 40, 50, 60], new)
        T = s["q"].shape[0]
        s["q"] = torch.nn.functional.pad(s["q"], (0, 0, 0, 0, 0, 3))
        s["seq"][1] = 2                              # fewer tokens than rows
        s["seq"][2] = s["table"].shape[1] * 16 + 1   # beyond the plan
        d = _dev(s)
        plan = _plan(s, max_new=plan_new)
        scratch = pb.alloc_scratch(plan)
        _call(s, d, plan, scratch)
        assert pb.check(scratch) == pb.DEVICE_CAPACITY
        out, lse = d["out"].cpu(), d["lse"].cpu()
        stay = list(range(s["qsl"][1], s["qsl"][3])) + list(range(T, T + 3))
        assert (out[stay] == 7).all() and (lse[stay] == 7).all()
        for b in (0, 3):
            one = ref.attend(s["q"][s["qsl"][b]:s["qsl"][b + 1]], s["k_cache"], s["v_cache"], s["k_scales"],
                             s["v_scales"], s["table"][b:b + 1], [s["seq"][b]], [0, new[b]], s["scale"])
            r = slice(s["qsl"][b], s["qsl"][b + 1])
            _close((out[r], lse[r]), one)


def test_more_rows_than_the_plan_holds():
    s = _problem(13, "int8", 8, 2, 64, 16, [30, 40], [2, 3])
    d = _dev(s)
    plan = _plan(s, max_new=2)
    scratch = pb.alloc_scratch(plan)
    _call(s, d, plan, scratch)
    assert pb.check(scratch) == pb.DEVICE_CAPACITY
    assert (d["out"][2:] == 7).all() and not (d["out"][:2] == 7).all()


@pytest.mark.parametrize("new", [[1, 1, 1], [3, 1, 2], [80, 70, 90]])
def test_pages_outside_the_pool_read_as_zeros(new):
    s = _problem(14, "e4m3", 8, 2, 128, 16, [100, 333, 50], new)
    s["table"][0, 2] = s["k_cache"].shape[0]
    s["table"][1, 5] = -3
    got = _run(s)
    assert got[2] == pb.DEVICE_PAGE_ID
    _close(got, _want(s))


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [4, 1, 2, 3], [70, 1, 80, 3]])
def test_strides(new):
    # halves of one allocation with heads outside slots; padded q, out and scales
    s = _problem(15, "int8", 8, 4, 128, 32, [100, 1, 64, 300], new, dirty=False)
    H, D, ps, pool = 4, 128, 32, s["k_cache"].shape[0]
    d = _dev(s)
    both = torch.zeros(pool, 2, H, ps, D, dtype=torch.int8, device="cuda")
    for i, n in enumerate(("k_cache", "v_cache")):
        v = both[:, i].transpose(1, 2)
        v.copy_(d[n])
        d[n] = v
    sc = torch.zeros(pool, 2 * H + 1, device="cuda")
    for i, n in enumerate(("k_scales", "v_scales")):
        v = sc[:, i * H:(i + 1) * H]
        v.copy_(d[n])
        d[n] = v
    T = s["q"].shape[0]
    for n in ("q", "out"):
        wide = torch.full((T, 10, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        wide[:, 1:9, :D] = d[n]
        d[n + "_all"] = wide
        d[n] = wide[:, 1:9, :D]
    plan = _plan(s)
    scratch = pb.alloc_scratch(plan)
    _call(s, d, plan, scratch)
    assert pb.check(scratch) == 0
    _close((d["out"].cpu(), d["lse"].cpu()), _want(s))
    edge = d["out_all"].clone()
    edge[:, 1:9, :D] = 7.0
    assert (edge == 7.0).all()


def test_rows_of_odd_alignment():
    # few rows need 4-byte rows only
    s = _problem(16, "int8", 8, 2, 64, 16, [100, 31], [2, 3])
    d = _dev(s)
    T = s["q"].shape[0]
    wide = torch.zeros(T, 8, 66, dtype=torch.bfloat16, device="cuda")
    wide[..., 2:] = d["q"]
    d["q"] = wide[..., 2:]
    d["out"] = torch.zeros(T, 8, 66, dtype=torch.bfloat16, device="cuda")[..., 2:]
    plan = _plan(s)
    scratch = pb.alloc_scratch(plan)
    _call(s, d, plan, scratch)
    _close((d["out"].cpu(), d["lse"].cpu()), _want(s))


def test_a_pool_beyond_32_bits():
    H, D, ps = 8, 256, 64
    pool = (1 << 32) // (H * D * ps) + 40
    s = _problem(17, "int8", 16, H, D, ps, [150, 90], [1, 2], dirty=False)
    n = s["k_cache"].shape[0]
    d = _dev(s)
    ids = torch.randperm(30)[:n] + pool - 30
    for name in ("k_cache", "v_cache"):
        big = torch.empty(pool, ps, H, D, dtype=torch.int8, device="cuda")
        big[ids.cuda()] = d[name]
        d[name] = big
    for name in ("k_scales", "v_scales"):
        big = torch.full((pool, H), math.nan, device="cuda")
        big[ids.cuda()] = d[name]
        d[name] = big
    d["table"] = torch.tensor([[int(ids[i]) if i < n else 0 for i in row] for row in s["table"].tolist()],
                              dtype=torch.int32, device="cuda")
    for new in (2, 70):                              # the split kernel, then the chunked one
        plan = _plan(s, max_new=new)
        scratch = pb.alloc_scratch(plan)
        _call(s, d, plan, scratch)
        assert pb.check(scratch) == 0 and plan.chunked == (new == 70)
        _close((d["out"].cpu(), d["lse"].cpu()), _want(s))


def test_one_long_context():
    s = _problem(18, "e4m3", 8, 2, 128, 16, [40000], [1])
    got = _run(s, decode=True)
    _close(got, _want(s, decode=True))


@pytest.mark.parametrize("new", [[1] * 5, [3, 1, 4, 2, 1], [70, 3, 90, 1, 66]])
def test_calls_repeat_bitwise_and_graphs_replay(new):
    s = _problem(20, "int8", 8, 2, 128, 16, [700, 3, 2000, 0, 90], new)
    plan = _plan(s, max_pages_per_seq=s["table"].shape[1])
    d = _dev(s)
    scratch = pb.alloc_scratch(plan)
    _call(s, d, plan, scratch)
    out, lse = d["out"].clone(), d["lse"].clone()
    _close((out.cpu(), lse.cpu()), _want(s))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _call(s, d, plan, scratch)
    for _ in range(3):
        d["out"].zero_()
        g.replay()
        assert torch.equal(d["out"], out) and torch.equal(d["lse"], lse)
    # shorter contexts and other queries in the same buffers
    s["seq"] = [max(n, L // 2) for L, n in zip(s["seq"], new)]
    s["q"] = s["q"].flip(0).contiguous()
    d["seq"].copy_(torch.tensor(s["seq"], dtype=torch.int32))
    d["q"].copy_(s["q"])
    g.replay()
    torch.cuda.synchronize()
    assert pb.check(scratch) == 0
    _close((d["out"].cpu(), d["lse"].cpu()), _want(s))


def test_two_streams_with_their_own_scratch():
    a = _problem(21, "int8", 8, 2, 128, 16, [700, 900, 2000], [1, 1, 1])
    b = _problem(22, "e4m3", 8, 2, 128, 16, [300, 90, 10], [80, 70, 66])
    runs = []
    for s in (a, b):
        plan = _plan(s)
        runs.append((s, _dev(s), plan, pb.alloc_scratch(plan), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, d, plan, scratch, stream in runs:
            with torch.cuda.stream(stream):
                _call(s, d, plan, scratch)
    torch.cuda.synchronize()
    for s, d, plan, scratch, stream in runs:
        assert pb.check(scratch) == 0
        _close((d["out"].cpu(), d["lse"].cpu()), _want(s))


def test_without_lse_and_without_rows():
    s = _problem(23, "int8", 8, 2, 64, 16, [40, 0], [2, 0])
    d = _dev(s)
    plan = _plan(s)
    scratch = pb.alloc_scratch(plan)
    d["lse"] = None
    _call(s, d, plan, scratch)
    s2 = _want(s)
    assert ((d["out"].cpu().double() - s2[0]).abs() <= s2[2]).all()
