"""pa_select_pages against the definition in 64 bits: the chosen pages have to be
equal, ties and near-ties included."""
import numpy as np
import pytest
import torch

from tests import long_refs as lr

pytestmark = pytest.mark.gpu
MARK = -77


@pytest.fixture(scope="module")
def pb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_12_gb300 import binding
    binding.load()
    return binding


def make(lens, Hq, Hkv, D, ps, *, top, first=1, last=2, rows=None, seed=0, spread=1.0, extra_rows=0):
    g = torch.Generator().manual_seed(seed)
    n_pages = [-(-L // ps) for L in lens]
    pool = sum(n_pages) + 3
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    W = max(max(n_pages), 1)
    bt = torch.full((len(lens), W), 2 ** 31 - 1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(n_pages):
        bt[b, :n] = perm[at:at + n]
        at += n
    k = torch.randn(pool, 4, Hkv, D, generator=g) * spread
    bounds = torch.stack([k.amin(1), k.amax(1)], 2).bfloat16()
    qsl = None if rows is None else np.concatenate([[0], np.cumsum(rows)]).tolist()
    T = len(lens) if rows is None else qsl[-1]
    q = torch.randn(T + extra_rows, Hq, D, generator=g).bfloat16()
    return dict(lens=list(lens), Hq=Hq, Hkv=Hkv, D=D, ps=ps, top=top, first=first, last=last, bt=bt, bounds=bounds, q=q,
                qsl=qsl, T=T + extra_rows, W=W)


def run(pb, d, *, max_total_q=None, stream=None, code=0, score_rows=None, max_pages=None):
    plan = pb.sparse_plan(num_q_heads=d["Hq"], num_kv_heads=d["Hkv"], head_dim=d["D"], page_size=d["ps"],
                          max_batch=len(d["lens"]), max_pages_per_seq=max_pages or d["W"],
                          max_total_q=max_total_q or d["T"], top_pages=d["top"], first_pages=d["first"],
                          last_pages=d["last"])
    if score_rows is not None:
        plan.score_rows = min(plan.score_rows, score_rows)
    scratch = pb.alloc_scratch(plan)
    pages = torch.full((d["T"], d["Hkv"], d["top"]), MARK, dtype=torch.int32, device="cuda")
    args = [x.cuda() for x in (d["q"], d["bounds"], d["bt"], torch.tensor(d["lens"], dtype=torch.int32))]
    qsl = None if d["qsl"] is None else torch.tensor(d["qsl"], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    pb.select_pages(plan, *args, pages, query_start_loc=qsl, scratch=scratch, stream=stream)
    assert pb.check(scratch, stream) == code
    torch.cuda.synchronize()
    return pages.cpu()


def check(d, got, skip=()):
    want = lr.select(d["q"], d["bounds"], d["bt"], d["lens"], page_size=d["ps"], num_kv_heads=d["Hkv"], top=d["top"],
                     first=d["first"], last=d["last"], query_start_loc=d["qsl"])
    for row in range(d["T"]):
        if row in want and row not in skip:
            assert torch.equal(got[row], want[row]), (row, got[row], want[row])
        else:
            assert (got[row] == MARK).all(), row


SHAPES = [(8, 2, 64, 16), (32, 8, 128, 16), (16, 8, 256, 32), (24, 8, 128, 64), (8, 8, 64, 64), (40, 2, 128, 16),
          (14, 2, 64, 32), (28, 4, 256, 16), (12, 1, 128, 16)]


@pytest.mark.parametrize("Hq,Hkv,D,ps", SHAPES)
def test_decode(pb, Hq, Hkv, D, ps):
    lens = [0, 1, ps, ps + 1, 8 * ps, 8 * ps + 1, 21 * ps - 1, 130 * ps + 5, 300 * ps]
    for top, first, last in ((8, 1, 2), (1, 0, 1), (5, 4, 1), (33, 0, 3)):
        d = make(lens, Hq, Hkv, D, ps, top=top, first=first, last=last, seed=Hq + top)
        check(d, run(pb, d))


@pytest.mark.parametrize("Hq,Hkv,D,ps", SHAPES)
def test_packed_rows(pb, Hq, Hkv, D, ps):
    # rows of one request lie on either side of the length from which a selection leaves pages out
    lens = [20 * ps + 3, 5, 0, 9 * ps + 1, 200 * ps + 7, 8 * ps + 2]
    rows = [37, 3, 0, 40, 5, 30]
    d = make(lens, Hq, Hkv, D, ps, top=9, rows=rows, seed=Hq, extra_rows=4)
    check(d, run(pb, d))


@pytest.mark.parametrize("Hq,D", [(128, 64), (96, 256), (65, 128)])
def test_large_groups(pb, Hq, D):
    d = make([70 * 16, 33 * 16 + 2], Hq, 1, D, 16, top=9, seed=Hq)
    check(d, run(pb, d))
    d = make([70 * 16, 33 * 16 + 2], Hq, 1, D, 16, top=9, rows=[3, 5], seed=Hq)
    check(d, run(pb, d))


def test_many_rows(pb):
    d = make([1300], 8, 2, 64, 16, top=6, rows=[700], seed=20)
    check(d, run(pb, d))


def test_long_context(pb):
    d = make([131071, 70000], 16, 2, 64, 16, top=128, last=4, seed=1)
    check(d, run(pb, d))
    d = make([65536 * 16], 4, 1, 64, 16, top=300, seed=2)          # the largest block table
    check(d, run(pb, d))


def test_several_passes_over_the_rows(pb):
    d = make([3000, 2000, 900], 8, 2, 64, 16, top=12, rows=[60, 31, 20], seed=3)
    want = run(pb, d)
    check(d, want)
    for n in (1, 7, 32):
        assert torch.equal(run(pb, d, score_rows=n), want)
    assert torch.equal(run(pb, d, max_total_q=500, max_pages=1000), want) if d["W"] >= 1000 else True


def test_exact_ties_go_to_the_lower_page(pb):
    # every page has the same bounds; then pages of two kinds; then a zero query
    d = make([400 * 16], 8, 2, 64, 16, top=40, seed=4)
    d["bounds"][:] = d["bounds"][0]
    check(d, run(pb, d))
    d["bounds"][::3] = d["bounds"][1]
    d["bounds"][1::3] *= 2
    check(d, run(pb, d))
    d["q"][:] = 0
    check(d, run(pb, d))


@pytest.mark.parametrize("n", [300, 1500])
def test_near_ties(pb, n):
    # scores that 32-bit sums cannot tell apart: one large dim common to all, tiny
    # differences in another.  300 undecided pages are ranked, 1500 searched.
    d = make([n * 16], 4, 1, 64, 16, top=50, seed=5)
    g = torch.Generator().manual_seed(6)
    b = torch.zeros_like(d["bounds"])
    b[:, :, :, 0] = 2.0 ** 20
    b[:, :, :, 1] = (1 + torch.rand(b.shape[0], 1, 1, generator=g)).bfloat16() * 2.0 ** -8
    d["bounds"] = b
    d["q"][:] = 1.0
    check(d, run(pb, d))
    d["q"][:, 2:] = -1.0
    check(d, run(pb, d))


def test_group_maximum(pb):
    # one head of the group decides, another for other pages
    d = make([900 * 16], 8, 1, 64, 16, top=30, seed=7)
    d["q"][0, 1:7] = 0
    check(d, run(pb, d))


def test_scales_of_values(pb):
    # subnormal bounds, small and large ones, and sums beyond the 32-bit range
    for s in (1e-39, 1e-38, 1e-30, 1e-19, 1e19, 3e37):
        d = make([500 * 16, 60 * 16], 8, 2, 64, 16, top=20, seed=8, spread=s)
        check(d, run(pb, d))
        if s < 1:
            d["q"] = (d["q"].double() / s * 1e-3).clamp(-1e38, 1e38).bfloat16()
            check(d, run(pb, d))
            d["q"] = (d["q"].double() * 1e-39).bfloat16()
            check(d, run(pb, d))


def test_infinities_and_nan(pb):
    d = make([200 * 16, 200 * 16], 8, 2, 64, 16, top=12, seed=9)
    d["bounds"][d["bt"][0, 50], 0, 1, 3] = float("inf")
    d["bounds"][d["bt"][0, 70], 0, 0, 3] = float("-inf")
    d["bounds"][d["bt"][0, 71], 1, 0, 3] = float("nan")
    for i in range(100, 130):                     # more than fit
        d["bounds"][d["bt"][1, i], 0, 0, 1] = float("nan")
    check(d, run(pb, d))
    d["q"][0, 2, 9] = float("nan")
    d["q"][1, 7, 9] = float("-inf")
    check(d, run(pb, d))


def test_bad_requests_are_untouched(pb):
    d = make([100 * 16, 50 * 16, 60 * 16], 8, 2, 64, 16, top=12, seed=10)
    d["lens"][1] = 100 * 16 + 1
    got = run(pb, d, code=pb.DEVICE_CAPACITY)
    d["lens"][1] = 50 * 16
    check(d, got, skip=(1,))
    d = make([100 * 16, 50, 60 * 16], 8, 2, 64, 16, top=12, rows=[3, 50, 4], seed=11)
    d["lens"][1] = 49
    got = run(pb, d, code=pb.DEVICE_CAPACITY)
    d["lens"][1] = 50
    check(d, got, skip=range(3, 53))


def test_page_outside_the_pool_scores_zero(pb):
    d = make([100 * 16], 8, 2, 64, 16, top=99, first=0, last=1, seed=12)
    n = d["bounds"].shape[0]
    page = int(d["bt"][0, 20])
    want = dict(d)
    d["bt"][0, 20] = n
    got = run(pb, d, code=pb.DEVICE_PAGE_ID)
    want["bounds"] = d["bounds"].clone()
    want["bounds"][page] = 0
    want["bt"] = d["bt"].clone()
    want["bt"][0, 20] = page
    check(want, got)


def test_random_problems(pb):
    rng = np.random.default_rng(13)
    for i in range(12):
        Hq, Hkv, D, ps = SHAPES[rng.integers(len(SHAPES))]
        B = int(rng.integers(1, 6))
        lens = rng.integers(0, 150 * ps, size=B)
        rows = None if i % 3 == 0 else [int(rng.integers(0, min(L, 20) + 1)) for L in lens]
        first, last = int(rng.integers(0, 3)), int(rng.integers(1, 4))
        top = first + last + int(rng.integers(0, 40))
        if rows is not None and sum(rows) == 0:
            continue
        d = make(lens.tolist(), Hq, Hkv, D, ps, top=top, first=first, last=last, rows=rows, seed=100 + i)
        check(d, run(pb, d))


def test_strided_inputs_graph_and_stream(pb):
    d = make([100 * 16, 50 * 16], 8, 2, 64, 16, top=12, seed=14)
    wide = torch.zeros(2, 11, 64, dtype=torch.bfloat16)
    wide[:, 2:10] = d["q"]
    side = torch.cuda.Stream()
    check(d, run(pb, d, stream=side))
    plan = pb.sparse_plan(num_q_heads=8, num_kv_heads=2, head_dim=64, page_size=16, max_batch=2, max_pages_per_seq=100,
                          max_total_q=2, top_pages=12)
    scratch = pb.alloc_scratch(plan)
    q = wide.cuda()[:, 2:10]
    bounds = torch.zeros(d["bounds"].shape[0], 3, 2, 64, dtype=torch.bfloat16, device="cuda")[:, 1:]
    bounds.copy_(d["bounds"])
    bt, lens = d["bt"].cuda(), torch.tensor(d["lens"], dtype=torch.int32, device="cuda")
    pages = torch.full((2, 2, 12), MARK, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pb.select_pages(plan, q, bounds, bt, lens, pages, scratch=scratch)
    for seed in (15, 16):
        e = make([100 * 16, 31 * 16], 8, 2, 64, 16, top=12, seed=seed)
        q.copy_(e["q"])
        bounds[:e["bounds"].shape[0]] = e["bounds"].cuda()
        bt.copy_(e["bt"])
        lens.copy_(torch.tensor(e["lens"], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check(e, pages.cpu())


@pytest.mark.parametrize("n", [300, 1500])
@pytest.mark.parametrize("D", [64, 256])
def test_finite_queries_whose_magnitudes_sum_past_the_32_bit_range(pb, n, D):
    # |q|_1 = D 2^124 is not a float, the scores are: near-ties that 32-bit sums cannot tell apart
    d = make([n * 16], 4, 1, D, 16, top=50, seed=30)
    g = torch.Generator().manual_seed(31)
    b = torch.zeros_like(d["bounds"])
    b[:, :, :, 0] = 2.0 ** -90
    b[:, :, :, 1] = (1 + torch.rand(b.shape[0], 1, 1, generator=g)).bfloat16() * 2.0 ** -118
    d["bounds"] = b
    d["q"][:] = 2.0 ** 124
    check(d, run(pb, d))
    d["q"][:, :, 2:] = -(2.0 ** 124)
    check(d, run(pb, d))
    # products near the end of the range: sums that overflow in 32 bits but not in 64
    sign = 1 - 2.0 * (torch.arange(D) % 2)
    b = (8 * sign * (1 + 2.0 ** -6 * torch.randint(0, 9, (b.shape[0], 1, 1, D), generator=g))).bfloat16()
    d["bounds"] = b.expand_as(d["bounds"]).contiguous()
    check(d, run(pb, d))
    # beside them one that is not finite
    d["q"][0, 2, 5] = float("inf")
    check(d, run(pb, d))


def test_largest_and_smallest_finite_queries(pb):
    for q in (3.3895313892515355e38, 2.0 ** -133, 2.0 ** -126):
        for s in (2.0 ** -100, 1.0, 2.0 ** 100):
            d = make([300 * 16], 8, 2, 128, 16, top=20, seed=32, spread=s)
            d["q"] = (torch.sign(d["q"].float()) * q).bfloat16()
            assert torch.isfinite(d["q"]).all() and (d["q"] != 0).all()
            check(d, run(pb, d))
