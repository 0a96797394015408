"""pa_page_bounds against the smallest and largest key values of every page,
exactly; pages without new tokens, unowned pages and bad requests untouched."""
import numpy as np
import pytest
import torch

from paged_kv_gqa_12_gb300 import workloads as wl
from tests import gpu_helpers as gh
from tests import long_refs as lr

pytestmark = pytest.mark.gpu
MARK = 123.0


@pytest.fixture(scope="module")
def pb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_12_gb300 import binding
    binding.load()
    return binding


def problem(lens, Hkv, D, ps, kv, seed, **kw):
    extra = dict(k_scale=0.05, v_scale=0.05) if kv == "fp8_e4m3" else {}
    return wl.build_problem("decode", num_q_heads=Hkv, num_kv_heads=Hkv, head_dim=D, page_size=ps, seq_lens=lens,
                            kv_dtype=kv, seed=seed, **{**extra, **kw})


def run(pb, p, d, qsl=None, scratch=None, k_scales=None, lens=None):
    bounds = torch.full((p.num_pages, p.num_kv_heads, 2, p.head_dim), MARK, dtype=torch.bfloat16, device="cuda")
    pb.page_bounds(d["k"], d["bt"], d["sl"] if lens is None else lens, bounds,
                   query_start_loc=None if qsl is None else torch.tensor(qsl, dtype=torch.int32, device="cuda"),
                   kv_dtype=pb.KV_FP8_E4M3 if p.kv_dtype == "fp8_e4m3" else pb.KV_BF16, k_scale=p.k_scale,
                   k_scales=k_scales, scratch=scratch)
    torch.cuda.synchronize()
    return bounds.cpu().double()


def host_k(p):
    return gh._t(np.ascontiguousarray(p.k_cache))


def check(p, got, pages, scales=None):
    ref = lr.bounds_of(host_k(p), p.block_table, p.seq_lens.tolist(), p.page_size, p.k_scale, scales)
    for page in range(p.num_pages):
        want = ref[page] if page in pages else torch.full_like(got[page], MARK)
        assert torch.equal(got[page], want), page


def owned(p, first=None):
    return {int(p.block_table[b, i]) for b, L in enumerate(p.seq_lens.tolist())
            for i in range(0 if first is None else first[b] // p.page_size, -(-L // p.page_size))}


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("Hkv,D,ps", [(2, 64, 16), (8, 128, 16), (8, 256, 32), (3, 64, 64), (1, 64, 16), (20, 256, 16)])
def test_every_page(pb, kv, Hkv, D, ps):
    p = problem([1, 16, 0, 17, 63, 300, 64], Hkv, D, ps, kv, seed=Hkv + D)
    check(p, run(pb, p, gh.upload(p)), owned(p))


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_new_tokens_alone(pb, kv):
    lens, new = [1, 16, 0, 17, 63, 300, 64, 40], [1, 1, 0, 2, 63, 45, 17, 0]
    p = problem(lens, 4, 128, 16, kv, seed=3)
    qsl = np.concatenate([[0], np.cumsum(new)]).tolist()
    first = [L - n if n else 10 ** 9 for L, n in zip(lens, new)]
    check(p, run(pb, p, gh.upload(p), qsl=qsl), owned(p, first))


def test_many_requests(pb):
    # more requests than a CTA lists at a time
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 70, size=700)
    p = problem(lens, 2, 64, 16, "bf16", seed=5)
    check(p, run(pb, p, gh.upload(p)), owned(p))


def test_interleaved_layout_and_request_scales(pb):
    p = problem([40, 100], 4, 64, 32, "bf16", seed=6, layout="interleaved")
    check(p, run(pb, p, gh.upload(p)), owned(p))
    p = problem([40, 100, 33], 4, 64, 32, "fp8_e4m3", seed=7)
    scales = torch.tensor([0.02, 1.5, -0.25])
    got = run(pb, p, gh.upload(p), k_scales=scales.cuda())
    check(p, got, owned(p), scales)


def test_signed_zero_infinity_and_nan(pb):
    p = problem([16, 32], 2, 64, 16, "bf16", seed=8)
    d = gh.upload(p)
    page = int(p.block_table[0, 0])
    d["k"][page, 3, 0, 5] = float("inf")
    d["k"][page, 4, 0, 6] = float("-inf")
    d["k"][page, 5, 1, 7] = float("nan")
    got = run(pb, p, d)
    assert got[page, 0, 1, 5] == float("inf") and got[page, 0, 0, 6] == float("-inf")
    assert got[page, 1, :, 7].isnan().all()
    assert got[page].isnan().sum() == 2
    p = problem([16], 2, 64, 16, "fp8_e4m3", seed=9)
    d = gh.upload(p)
    page = int(p.block_table[0, 0])
    d["k"][page, 5, 1, 7] = 0x7F
    got = run(pb, p, d)
    assert got[page, 1, :, 7].isnan().all() and got[page].isnan().sum() == 2


def test_bad_requests_are_passed_over(pb):
    p = problem([40, 100, 33], 2, 64, 16, "bf16", seed=10)
    d = gh.upload(p)
    scratch = torch.zeros(pb.SCRATCH_HEADER_BYTES, dtype=torch.uint8, device="cuda")
    W = p.block_table.shape[1]
    got = run(pb, p, d, scratch=scratch, lens=torch.tensor([40, W * 16 + 1, 33], dtype=torch.int32, device="cuda"))
    assert pb.check(scratch) == pb.DEVICE_CAPACITY
    q = problem([40, 100, 33], 2, 64, 16, "bf16", seed=10)
    other = {int(x) for x in p.block_table[1, :7]}
    check(q, got, owned(q) - other)
    got = run(pb, p, d, scratch=scratch, qsl=[0, 41, 41, 42])      # 41 new tokens of 40
    assert pb.check(scratch) == pb.DEVICE_CAPACITY
    check(q, got, {int(p.block_table[2, 2])})
    d["bt"][1, 2] = p.num_pages
    d["bt"][2, 1] = -1
    got = run(pb, p, d, scratch=scratch)
    assert pb.check(scratch) == pb.DEVICE_PAGE_ID
    check(q, got, owned(q) - {int(p.block_table[1, 2]), int(p.block_table[2, 1])})


def test_strided_bounds_and_far_pages(pb):
    # a pool whose element offsets pass 32 bits, and bounds that are part of a wider array
    Hkv, D, ps = 8, 128, 16
    pages = (1 << 31) // (ps * Hkv * D) + 64
    k = torch.zeros(pages, ps, Hkv, D, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([[0, pages - 1, pages - 30]], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(1)
    rows = torch.randn(3, ps, Hkv, D, generator=g).bfloat16()
    k[ids[0].long()] = rows.cuda()
    wide = torch.zeros(pages, Hkv, 3, D, dtype=torch.bfloat16, device="cuda")
    bounds = wide[:, :, :2]
    pb.page_bounds(k, ids, torch.tensor([3 * ps - 4], dtype=torch.int32, device="cuda"), bounds)
    got = bounds[ids[0].long()].cpu()
    assert torch.equal(got[:2, :, 0], rows[:2].amin(1)) and torch.equal(got[:2, :, 1], rows[:2].amax(1))
    assert torch.equal(got[2, :, 0], rows[2, :ps - 4].amin(0)) and torch.equal(got[2, :, 1], rows[2, :ps - 4].amax(0))
    assert not wide[:, :, 2].any()


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("Hkv,D,ps,lo,hi,batch", [(20, 256, 16, 0, 150, 300), (2, 64, 16, 300, 1000, 330),
                                                  (1, 128, 64, 2000, 4000, 270)])
@pytest.mark.parametrize("fresh", [False, True])
def test_more_groups_of_pages_than_ctas(pb, kv, Hkv, D, ps, lo, hi, batch, fresh):
    """Each CTA takes several groups of pages, over more requests than it lists at a time."""
    rng = np.random.default_rng(D + batch)
    lens = rng.integers(lo, hi, size=batch)
    n = -(-lens // ps)
    pool = int(n.sum()) + 5
    g = torch.Generator(device="cuda").manual_seed(D)
    k = torch.randn(pool, ps, Hkv, D, generator=g, device="cuda").bfloat16()
    if kv == "fp8_e4m3":
        k = k.to(torch.float8_e4m3fn).view(torch.uint8)
    table = torch.full((batch, int(n.max())), -1, dtype=torch.int32)
    perm = torch.from_numpy(rng.permutation(pool)[:int(n.sum())].astype(np.int32))
    filled = torch.zeros(pool, dtype=torch.int64)          # filled slots of the pages that are to be written
    new = rng.integers(0, lens + 1) if fresh else lens
    at = 0
    for b in range(batch):
        table[b, :n[b]] = perm[at:at + n[b]]
        if new[b]:
            first = (lens[b] - new[b]) // ps
            ids = table[b, first:n[b]].long()
            filled[ids] = ps
            filled[ids[-1]] = int(lens[b] - (n[b] - 1) * ps)
        at += n[b]
    bounds = torch.full((pool, Hkv, 2, D), MARK, dtype=torch.bfloat16, device="cuda")
    qsl = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda() if fresh else None
    scratch = torch.zeros(pb.SCRATCH_HEADER_BYTES, dtype=torch.uint8, device="cuda")
    pb.page_bounds(k, table.cuda(), torch.from_numpy(lens.astype(np.int32)).cuda(), bounds, query_start_loc=qsl,
                   kv_dtype=pb.KV_FP8_E4M3 if kv == "fp8_e4m3" else pb.KV_BF16, k_scale=0.5, scratch=scratch)
    assert pb.check(scratch) == 0
    x = k.float() if kv == "bf16" else (k.view(torch.float8_e4m3fn).float() * 0.5).bfloat16().float()
    f = filled.cuda()
    out = (torch.arange(ps, device="cuda") >= f[:, None])[..., None, None]
    want = torch.stack([x.masked_fill(out, float("inf")).amin(1), x.masked_fill(out, -float("inf")).amax(1)], 2)
    want = torch.where((f > 0)[:, None, None, None], want, torch.full_like(want, MARK))
    assert torch.equal(bounds.float(), want)
