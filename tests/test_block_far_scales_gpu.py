"""pa_block_attend over pages whose V scales lie as far apart as the header allows: those of zeros, which count as 2^-100,
beside large ones.  Every key weighs the same, so a row's LSE is the logarithm of their number."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from paged_kv_gqa_12_gb300 import binding as pb  # noqa: E402

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.mark.parametrize("code", [pb.CODE_INT8, pb.CODE_E4M3])
@pytest.mark.parametrize("rows", [1, 3, 70])
@pytest.mark.parametrize("large", [0, 20, 25])
@pytest.mark.parametrize("ctas", [0, 1])
def test_zeros_beside_large_values(code, rows, large, ctas):
    Hq, Hkv, D, ps, pages = 8, 2, 64, 16, 40
    L, dt = pages * ps, torch.int8 if code == pb.CODE_INT8 else torch.uint8
    kc = torch.zeros(2, ps, Hkv, D, dtype=dt, device="cuda")
    vc = torch.full((2, ps, Hkv, D), 1 if code == pb.CODE_INT8 else 0x38, dtype=dt, device="cuda")      # 1
    ks, vs = torch.ones(2, Hkv, device="cuda"), torch.zeros(2, Hkv, device="cuda")
    vs[1] = 2.0 ** large
    table = (torch.arange(pages, dtype=torch.int32, device="cuda") % 4 == 1).to(torch.int32).view(1, pages)     # a quarter
    q = torch.randn(rows, Hq, D, device="cuda").bfloat16()
    plan = pb.block_plan(num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=ps, code=code, max_batch=1,
                         max_pages_per_seq=pages, max_total_q=rows, max_new=rows, num_ctas=ctas)
    assert plan.chunked == (rows == 70)
    scratch = pb.alloc_scratch(plan)
    out, lse = torch.empty_like(q), torch.empty(rows, Hq, device="cuda")
    pb.block_attend(plan, q, kc, vc, ks, vs, table, torch.tensor([L], dtype=torch.int32, device="cuda"),
                    query_start_loc=torch.tensor([0, rows], dtype=torch.int32, device="cuda"), scale=1.0, out=out,
                    lse=lse, scratch=scratch)
    assert pb.check(scratch) == 0
    n = torch.arange(L - rows + 1, L + 1).double()
    big = torch.stack([(table[0].cpu().repeat_interleave(ps)[:int(k)]).sum() for k in n]).double()
    # logarithms of numbers up to 2^7 rounded by 2^-18 a few times; weights and denominators to fp32's step or 2^-16 where
    # they are subnormal
    tol = 2.0 ** -14
    assert ((lse.cpu().double() - torch.log(n)[:, None]).abs() <= tol).all(), float((lse.cpu().double() - torch.log(n)[:, None]).abs().max())
    want = (big / n * 2.0 ** large)[:, None, None]
    assert ((out.cpu().double() - want).abs() <= want * (2.0 ** -8 + 2.0 ** -11 + 2 * tol)).all()
    assert math.isfinite(float(lse.sum()))
