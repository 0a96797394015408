"""pa_block_attend where a head's V scales are all 0 (an empty cache, a head that is padding) or near 0 and contexts are
long: the denominator sums a weight over its V scale for each key."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from paged_kv_gqa_12_gb300 import binding as pb  # noqa: E402

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

PS = 64


def _run(L, rows, code, v_scale, sinks, first=0.0, **plan_kw):
    """One request of L keys and `rows` rows, 8 q and 2 kv heads of 64.  A row's scores are `first` below 1 for the
    first 64 keys and 1 for the others.  -> (out, lse, wanted lse) with the device's code checked."""
    Hq, Hkv, D, pages = 8, 2, 64, -(-L // PS)
    kinds = dict(dtype=torch.int8 if code == pb.CODE_INT8 else torch.uint8, device="cuda")
    one = 1 if code == pb.CODE_INT8 else 0x38                    # the code of 1
    kc = torch.zeros(2, PS, Hkv, D, **kinds)
    kc[:, :, :, 0] = one
    vc = torch.full((2, PS, Hkv, D), 127 if code == pb.CODE_INT8 else 0x7e, **kinds)     # (0x7e: 448)
    ks, vs = torch.ones(2, Hkv, device="cuda"), torch.full((2, Hkv), v_scale, device="cuda")
    ks[0] = 1.0 - first
    table = torch.ones(1, pages, dtype=torch.int32, device="cuda")
    table[0, 0] = 0
    q = torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    sk = torch.linspace(-3.0, 12.0, Hq, device="cuda") if sinks else None
    plan = pb.block_plan(num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=PS, code=code, max_batch=1,
                         max_pages_per_seq=pages, max_total_q=rows, max_new=rows, has_sinks=sinks, **plan_kw)
    scratch = pb.alloc_scratch(plan)
    out, lse = torch.full_like(q, 7.0), torch.full((rows, Hq), 7.0, device="cuda")
    pb.block_attend(plan, q, kc, vc, ks, vs, table, torch.tensor([L], dtype=torch.int32, device="cuda"),
                    query_start_loc=torch.tensor([0, rows], dtype=torch.int32, device="cuda"), scale=1.0, out=out,
                    lse=lse, sinks=sk, scratch=scratch)
    assert pb.check(scratch) == 0
    n = torch.arange(L - rows + 1, L + 1).double()               # keys of each row
    near = torch.log((n - PS) * math.e + PS * math.exp(1.0 - first))
    want = near[:, None].expand(rows, Hq)
    share = torch.ones_like(want)                                # of the keys, beside the sink
    if sinks:
        s = sk.cpu().double()[None, :].expand(rows, Hq)
        full = torch.logaddexp(want, s)
        want, share = full, torch.exp(want - full)
    return out.cpu().double(), lse.cpu().double(), want, share, plan


def _close(got, L, v_scale, code):
    out, lse, want, share, _ = got
    # a share adds at most L / 16 numbers to a row's sum (L / 64 in chunks), each addition off by half a step, and some
    # more where lanes, warps and parts meet; scores beside the logarithm of a V scale, maxima, and their sums with the
    # denominator's logarithm are numbers below 128 in units of log 2, each rounded by at most 2^-18 (five of them), and
    # an exponential or logarithm is good to 2^-20
    tol = (L / 16 + 64) * 2.0 ** -24 + 2.0 ** -15
    assert lse.isfinite().all() and ((lse - want).abs() <= tol).all(), float((lse - want).abs().max())
    # every V is the same: scales below 2^-100 count as 2^-100; the weights are off by half a step of f16, the output of bf16
    v = (127 if code == pb.CODE_INT8 else 448) * max(v_scale, 2.0 ** -100)
    assert ((out - v * share[..., None]).abs() <= v * (2.0 ** -11 + 2.0 ** -8 + 2 * tol) + 2.0 ** -126).all(), float(out.abs().max())


@pytest.mark.parametrize("code", [pb.CODE_INT8, pb.CODE_E4M3])
@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("v_scale", [0.0, 2.0 ** -90])
@pytest.mark.parametrize("ctas", [1, 2, 0])
@pytest.mark.parametrize("rows", [1, 3])
def test_few_rows(code, sinks, v_scale, ctas, rows):
    L = 40000 if v_scale == 0 else 1 << 19                       # 2^14 / 2^-90 a key: past 2^128 from 2^24 keys
    got = _run(L, rows, code, v_scale, sinks, num_ctas=ctas)
    assert got[4].chunked == 0
    _close(got, L, v_scale, code)


@pytest.mark.parametrize("code", [pb.CODE_INT8, pb.CODE_E4M3])
@pytest.mark.parametrize("sinks", [False, True])
def test_chunks(code, sinks):
    # the first 64 keys set a maximum that the others stay less than 2^8 above
    L, rows = 40000, 70
    got = _run(L, rows, code, 0.0, sinks, first=7.9 * math.log(2.0))
    assert got[4].chunked == 1
    _close(got, L, 0.0, code)
