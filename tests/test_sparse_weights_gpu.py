"""Softmax weights of pa_sparse_attend beyond one bf16: weights that one bf16 rounds
all the same way, where values cancel, and infinite values."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_12_gb300 import binding
    binding.load()
    return binding


def attend(pb, q, k, v, L, *, scale, splits, sinks=None):
    """One request whose pages lie in order, every page chosen."""
    n, ps, Hkv, D = k.shape
    e4m3 = k.dtype == torch.uint8
    plan = pb.sparse_plan(num_q_heads=q.shape[1], num_kv_heads=Hkv, head_dim=D, page_size=ps,
                          kv_dtype=pb.KV_FP8_E4M3 if e4m3 else pb.KV_BF16, max_batch=1, max_pages_per_seq=n,
                          max_total_q=1, top_pages=n, first_pages=0, last_pages=1, num_splits=splits,
                          has_sinks=sinks is not None)
    scratch = pb.alloc_scratch(plan)
    pages = torch.arange(n, dtype=torch.int32, device="cuda").expand(1, Hkv, n).contiguous()
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(q.shape[:2], device="cuda")
    pb.sparse_attend(plan, q.cuda(), k.cuda(), v.cuda(), torch.arange(n, dtype=torch.int32, device="cuda")[None],
                     torch.tensor([L], dtype=torch.int32, device="cuda"), pages, scale=scale, out=out, lse=lse,
                     sinks=None if sinks is None else sinks.cuda(), scratch=scratch)
    assert pb.check(scratch) == 0
    return out.cpu()[0], lse.cpu()[0]


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("group", [4, 16])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,ps", [(64, 16), (64, 64), (128, 16), (256, 32)])
def test_equal_weights_between_two_bf16(pb, D, ps, kv, group, splits):
    """Every other key has the weight 1/2 + 2^-9, halfway between two bf16, and the values of the two kinds of keys
    nearly cancel: what a rounding of the weights leaves is as large as the output.

    Tolerance: half a bf16 step of the output; the weights' second bf16 leaves at most 2^-15 of a weight; a score is
    one product, and its 32-bit scaling and exponential are off by less than 2^-20; at most 1024 / 4 products a warp
    are added in 32 bits, each addition off by at most 2^-23 of the sum of magnitudes: 2^-15.  Together below 2^-13
    of the sum of weight x |value|.  The log-sum-exp: 256 additions of at most 2^-24 and the rest 2^-20, below 2^-15."""
    p2 = 0.5 + 2.0 ** -9
    for n in (1, 2, 7, 1024 // ps):
        L = n * ps
        k = torch.zeros(n, ps, 1, D)
        v = torch.zeros(n, ps, 1, D)
        k[:, 1::2, :, 0] = -1.0
        size = 2.0 ** (torch.arange(D) % 7 - 3) * (1 - 2.0 * (torch.arange(D) % 2))
        v[:, 0::2] = -0.5 * size
        v[:, 1::2] = size
        q = torch.zeros(1, group, D)
        q[:, :, 0] = 1.0
        q = q.bfloat16()
        dt = (lambda x: x.to(torch.float8_e4m3fn).view(torch.uint8)) if kv == "e4m3" else (lambda x: x.bfloat16())
        scale = float(torch.tensor(-math.log(p2), dtype=torch.float32))
        out, lse = attend(pb, q, dt(k), dt(v), L, scale=scale, splits=splits)
        w = math.exp(-scale)
        o = (w - 0.5) / (1 + w) * size.double()
        spread = (w + 0.5) / (1 + w) * size.double().abs()
        err = (out.double() - o).abs()
        assert (err <= 2.0 ** -8 * o.abs() + 2.0 ** -13 * spread).all(), (n, (err / spread).max())
        assert (lse.double() - math.log(L / 2 * (1 + w))).abs().max() < 2.0 ** -15


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("D,ps,group", [(64, 16, 4), (128, 16, 8), (256, 32, 4), (128, 64, 16)])
def test_infinite_values(pb, D, ps, group, splits):
    """An attended value of +-infinity makes its dim of the output that infinity (both, or a NaN: NaN), on whole pages
    and on one that the context ends in, and no other dim or head changes a bit."""
    g = torch.Generator().manual_seed(D)
    n = 40
    L = n * ps - 7
    k, v = (torch.randn(n, ps, 2, D, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(1, 2 * group, D, generator=g).bfloat16()
    sinks = torch.randn(2 * group, generator=g)
    clean, _ = attend(pb, q, k, v, L, scale=D ** -0.5, splits=splits, sinks=sinks)
    inf = float("inf")
    put = {3: [(5, 2, inf)], 8: [(n - 1, 1, inf)], 17: [(0, 0, -inf)], 30: [(n - 1, ps - 8, -inf)],
           41: [(20, 3, inf), (21, 9, inf)], 50: [(7, 1, inf), (30, 4, -inf)], 63: [(11, 6, float("nan"))]}
    for d, cells in put.items():
        for page, slot, x in cells:
            v[page, slot, 1, d] = x
    v[n - 1, ps - 7:, :, 5] = inf                 # behind the end: not attended
    out, _ = attend(pb, q, k, v, L, scale=D ** -0.5, splits=splits, sinks=sinks)
    assert torch.equal(out[:group], clean[:group])
    rest = [d for d in range(D) if d not in put]
    assert torch.equal(out[group:, rest], clean[group:, rest])
    for d, want in ((3, inf), (8, inf), (17, -inf), (30, -inf), (41, inf)):
        assert (out[group:, d] == want).all(), (d, out[group:, d])
    assert out[group:, [50, 63]].isnan().all()


def test_weights_that_are_powers_of_two_and_zero(pb):
    """Weights that one bf16 holds (1, and the 2^-20 of far keys) with infinite values, and far keys whose weight is
    exactly zero beside finite ones."""
    D, ps = 64, 16
    k = torch.zeros(4, ps, 1, D)
    k[2:, :, 0, 0] = -20.0
    v = torch.ones(4, ps, 1, D)
    v[1, 4, 0, 7] = float("inf")
    v[3, 2, 0, 9] = float("-inf")
    q = torch.zeros(1, 4, D)
    q[:, :, 0] = 1.0
    out, _ = attend(pb, q.bfloat16(), k.bfloat16(), v.bfloat16(), 64, scale=math.log(2.0), splits=1)
    rest = [d for d in range(D) if d not in (7, 9)]
    assert (out[:, 7] == float("inf")).all() and (out[:, 9] == float("-inf")).all() and (out[:, rest] == 1).all()
    v[3, 2, 0, 9] = v[1, 4, 0, 7] = 1.0
    k[2:, :, 0, 0] = -3000.0                      # 2^-3000: zero
    v[2:] = 500.0
    out, _ = attend(pb, q.bfloat16(), k.bfloat16(), v.bfloat16(), 64, scale=math.log(2.0), splits=1)
    assert (out == 1).all()
