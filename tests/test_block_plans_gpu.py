"""Calls of pa_block_attend whose plan's form the sizes decide: decode of large groups, chunks of more rows than planned."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from paged_kv_gqa_12_gb300 import binding as pb  # noqa: E402

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests import block_refs as ref  # noqa: E402
from tests import test_block_attend_gpu as at  # noqa: E402


@pytest.mark.parametrize("kind,Hq,Hkv,D,batch", [("int8", 64, 1, 64, 304), ("int8", 71, 1, 64, 512), ("e4m3", 128, 1, 128, 400),
                                                 ("int8", 128, 2, 256, 152), ("e4m3", 49, 1, 128, 65535)])
def test_decode_of_large_groups_planned_for_many_requests(kind, Hq, Hkv, D, batch):
    lens = [33, 0, 1, 500, 64]
    s = at._problem(Hq, kind, Hq, Hkv, D, 16, [max(0, L - 1) for L in lens], [1 if L else 0 for L in lens], sinks=True)
    s["q"] = torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(3)).bfloat16()
    plan = at._plan(s, max_batch=batch, max_total_q=batch)
    got = at._run(s, decode=True, plan=plan)
    assert got[2] == 0 and plan.chunked == 0
    at._close(got, ref.attend(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"], s["seq"], None,
                              s["scale"], sinks=s["sinks"]))


@pytest.mark.parametrize("group", [0, 1])
def test_more_rows_than_a_chunked_plan_holds(group):
    new = [40, 70, 60, 61, 3]
    s = at._problem(13, "int8", 8, 2, 64, 16, [30, 40, 0, 5, 9], new)
    if group:                                        # requests attended one at a time
        wide = torch.zeros(5, 1 << 18, dtype=torch.int32)
        wide[:, :s["table"].shape[1]] = s["table"]
        s["table"] = wide
    d = at._dev(s)
    plan = at._plan(s, max_new=60)
    assert plan.chunked == 1 and (plan.group_requests == 1) == bool(group)
    scratch = pb.alloc_scratch(plan)
    at._call(s, d, plan, scratch)
    assert pb.check(scratch) == pb.DEVICE_CAPACITY
    out, lse = d["out"].cpu(), d["lse"].cpu()
    for b, n in enumerate(new):
        r = slice(s["qsl"][b], s["qsl"][b + 1])
        if n > 60:
            assert (out[r] == 7).all() and (lse[r] == 7).all()
        else:
            one = ref.attend(s["q"][r], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"][b:b + 1],
                             [s["seq"][b]], [0, n], s["scale"], chunked=True)
            at._close((out[r], lse[r]), one, b)
