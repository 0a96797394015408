"""Calls of pa_block_attend whose plan's form the sizes decide: decode of large groups."""
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
