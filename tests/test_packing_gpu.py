"""Packings whose entries lie so far apart that their differences wrap: the requests beside the wrap are refused, the
others answered, nothing else is written."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from paged_kv_gqa_12_gb300 import binding as pb  # noqa: E402

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests import block_refs as ref  # noqa: E402
from tests import test_append_blocks_gpu as ap  # noqa: E402
from tests import test_block_attend_gpu as at  # noqa: E402

FAR = [2 ** 31 - 1, -2 ** 31]                        # from one to the other: 1, in arithmetic that wraps


def _qsl(n):
    return torch.tensor([0, n] + FAR, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n", [3, 70])
def test_block_attend(n):
    s = at._problem(1, "int8", 8, 2, 64, 16, [30, 40, 50], [n, 2, 1])
    d = at._dev(s)
    d["qsl"] = _qsl(n)
    plan = at._plan(s)
    assert plan.chunked == (n == 70)
    scratch = pb.alloc_scratch(plan)
    at._call(s, d, plan, scratch)
    assert pb.check(scratch) == pb.DEVICE_CAPACITY
    out, lse = d["out"].cpu(), d["lse"].cpu()
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()
    at._close((out[:n], lse[:n]), ref.attend(s["q"][:n], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                             s["table"][:1], s["seq"][:1], [0, n], s["scale"], chunked=n == 70))


def test_extend():
    B, ps, W, Hq, Hkv, D, n = 3, 16, 8, 8, 2, 64, 40
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(B * W, ps, Hkv, D, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(n + 3, Hq, D, generator=g).bfloat16()
    plan = pb.plan(mode=pb.MODE_EXTEND, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=ps, max_batch=B,
                   max_pages_per_seq=W, max_total_q=n + 3)
    scratch = pb.alloc_scratch(plan)
    out, lse = torch.full_like(q, 7.0).cuda(), torch.full((n + 3, Hq), 7.0, device="cuda")
    table = torch.arange(B * W, dtype=torch.int32, device="cuda").view(B, W)

    def call(qsl, batch):
        pb.extend(plan, q.cuda(), k.cuda(), v.cuda(), table[:batch], torch.tensor([60, 90, 80][:batch], dtype=torch.int32, device="cuda"),
                  qsl, scale=D ** -0.5, out=out, lse=lse, scratch=scratch)
    call(_qsl(n), 3)
    assert pb.check(scratch) == pb.DEVICE_CAPACITY
    got = out.clone(), lse.clone()
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()
    call(_qsl(n)[:2], 1)
    assert pb.check(scratch) == 0
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)


def test_append():
    s = ap._problem(3, "int8", 2, 64, 16, [20, 30, 40], [5, 2, 1])
    want, code = ap._run(s)
    assert code == 0
    keep = dict(s)
    keep["qsl"] = [0, 5] + FAR
    got, code = ap._run(keep)
    assert code == pb.DEVICE_CAPACITY
    pages = [int(x) for x in s["table"][0, :2]]
    others = [i for i in range(s["k_cache"].shape[0]) if i not in pages]
    for name in ("k_cache", "v_cache", "k_scales", "v_scales"):
        assert torch.equal(got[name][pages], want[name][pages])
        assert torch.equal(got[name][others], s[name][others])


def test_verify():
    V = 300
    p = torch.softmax(torch.randn(6, V, generator=torch.Generator().manual_seed(4)), -1)
    tokens = torch.tensor([0, 5, 9, 2, 3, 4], dtype=torch.int32)
    u, w = torch.full((6,), 0.3), torch.tensor([0.5, 0.5, 0.5])
    out = torch.full((3, 8), 99, dtype=torch.int32, device="cuda")
    num = torch.full((3,), 99, dtype=torch.int32, device="cuda")
    scratch = torch.zeros(pb.SCRATCH_HEADER_BYTES, dtype=torch.uint8, device="cuda")
    pb.verify_tokens(tokens.cuda(), p.cuda(), _qsl(3), u.cuda(), w.cuda(), out, num, scratch=scratch)
    assert pb.check(scratch) == pb.DEVICE_CAPACITY
    o, k = ref.verify(tokens, p, None, [0, 3], u, w, 8)
    assert torch.equal(out[:1].cpu(), o) and num[0] == k[0] and (out[1:] == 99).all() and (num[1:] == 99).all()
