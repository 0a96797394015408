"""pa_select_pages in every form its threads per row take, and sums that 32 bits get
wrong: a plan for one SM counts eight (row, kv head) pairs as many, so a few rows reach
the forms that a chunk of new tokens over a long context takes."""
import pytest
import torch

from tests import test_select_gpu as ts

pytestmark = pytest.mark.gpu
pb = ts.pb

# pages of a context for each form of many rows (one warp up to 512 pages, sixteen up to
# 8192, beyond which scores are read again), and of few
MANY = {300: 32, 600: 64, 1500: 128, 3000: 256, 6000: 512, 9000: 512}
FEW = {300: 64, 1500: 256, 3000: 1024, 9000: 1024}


def run(pb, d, many):
    plan = pb.sparse_plan(num_q_heads=d["Hq"], num_kv_heads=d["Hkv"], head_dim=d["D"], page_size=d["ps"],
                          max_batch=len(d["lens"]), max_pages_per_seq=d["W"], max_total_q=d["T"], top_pages=d["top"],
                          first_pages=d["first"], last_pages=d["last"], num_sms=1 if many else 0)
    assert d["T"] * d["Hkv"] >= 8 if many else d["T"] * d["Hkv"] < 8 * plan.shape.num_sms
    scratch = pb.alloc_scratch(plan)
    pages = torch.full((d["T"], d["Hkv"], d["top"]), ts.MARK, dtype=torch.int32, device="cuda")
    pb.select_pages(plan, d["q"].cuda(), d["bounds"].cuda(), d["bt"].cuda(),
                    torch.tensor(d["lens"], dtype=torch.int32, device="cuda"), pages,
                    query_start_loc=torch.tensor(d["qsl"], dtype=torch.int32, device="cuda"), scratch=scratch)
    assert pb.check(scratch) == 0
    return pages.cpu()


def cases():
    return [(True, n) for n in MANY] + [(False, n) for n in FEW]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("many,n", cases())
def test_random_scores(pb, D, many, n):
    for top in (7, n // 3):
        d = ts.make([n * 16 - 5, 20 * 16], 6, 2, D, 16, top=top, rows=[4, 1], seed=n + top)
        ts.check(d, run(pb, d, many))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("many,n", cases())
def test_ties_infinities_and_nan(pb, D, many, n):
    d = ts.make([n * 16], 4, 2, D, 16, top=n // 4, rows=[4], seed=n)
    d["bounds"][::3] = d["bounds"][1]
    d["bounds"][1::3] = d["bounds"][2]
    ts.check(d, run(pb, d, many))
    d["bounds"][d["bt"][0, n // 2].long(), 0, 1, 3] = float("inf")
    d["bounds"][d["bt"][0, n // 3].long(), 1, 0, 4] = float("nan")
    ts.check(d, run(pb, d, many))
    d["bounds"][d["bt"][0, n // 5: n - 3].long(), 0, 1, 5] = float("inf")      # more than fit
    ts.check(d, run(pb, d, many))
    d["bounds"][:] = d["bounds"][0]
    ts.check(d, run(pb, d, many))
    d["q"][:, 0] = float("nan")
    d["q"][:, 1:] = 0
    ts.check(d, run(pb, d, many))


def near_ties(n, m, D, *, rows):
    """A context of n pages of which m, spread over it, have scores within 2^-28 of one another; the others' lie far
    below."""
    d = ts.make([n * 16], 4, 2, D, 16, top=50, rows=[rows], seed=m)
    g = torch.Generator().manual_seed(n + m)
    b = torch.zeros_like(d["bounds"])
    at = d["bt"][0, torch.randperm(n - 3, generator=g)[:m].sort().values + 1].long()
    b[at, :, :, 0] = 2.0 ** 20
    b[at, :, :, 1] = (1 + torch.rand(m, 1, 1, generator=g)).bfloat16() * 2.0 ** -8
    d["bounds"] = b
    d["q"][:] = 1.0
    d["q"][1:, :, 2:] = -1.0
    return d


@pytest.mark.parametrize("many,n,cap", [(True, 300, 64), (True, 600, 128), (True, 1500, 256), (True, 3000, 512),
                                        (True, 6000, 512), (True, 9000, 512), (False, 300, 128), (False, 1500, 512),
                                        (False, 3000, 512)])
def test_undecided_pages_ranked_and_searched(pb, many, n, cap):
    # as many as the list in shared memory holds, one fewer and more; beyond it they are searched
    for m in (cap - 1, cap, cap + 1, cap + 30):
        if m < n - 3:
            ts.check((d := near_ties(n, m, 64, rows=4)), run(pb, d, many))
    for D in (128, 256):
        ts.check((d := near_ties(n, cap + 9, D, rows=4)), run(pb, d, many))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("many", [False, True])
def test_sums_of_alternating_sign(pb, D, many):
    """Half of the dims carry +-1 .. 2 that cancel exactly, the other half differences of 2^-22 and less that decide:
    32-bit sums lose them in an order of their own."""
    for n, seed in ((300, 1), (700, 2)):
        d = ts.make([n * 16], 4, 2, D, 16, top=40, rows=[4], seed=seed)
        g = torch.Generator().manual_seed(seed)
        b = torch.zeros(d["bounds"].shape[0], 2, D)
        big = (1 + torch.rand(b.shape[0], 2, D // 4, generator=g)).bfloat16().float()
        b[..., 0:D // 2:2], b[..., 1:D // 2:2] = big, -big
        b[..., D // 2:] = torch.randn(b.shape[0], 2, D // 2, generator=g) * 2.0 ** -22
        b = b[..., torch.randperm(D, generator=g)]
        d["bounds"] = b.bfloat16()[:, :, None].expand(-1, -1, 2, -1).contiguous()
        d["q"][:] = 1.0
        ts.check(d, run(pb, d, many))
        d["q"][:, 1] = -1.0
        ts.check(d, run(pb, d, many))


def test_capacities_beyond_the_call(pb):
    # a plan for more rows and wider block tables than the call has; entries behind a context are never read
    d = ts.make([3000, 2000, 900], 8, 2, 64, 16, top=12, rows=[60, 31, 20], seed=3)
    want = ts.run(pb, d)
    wide = torch.full((3, 1000), 2 ** 31 - 1, dtype=torch.int32)
    wide[:, :d["W"]] = d["bt"]
    d["bt"] = wide
    got = ts.run(pb, d, max_total_q=500, max_pages=1000)
    assert torch.equal(got, want)
    ts.check(d, got)
