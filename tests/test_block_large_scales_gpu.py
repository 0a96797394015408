"""pa_block_attend where V is next to the largest numbers that bf16 holds."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from paged_kv_gqa_12_gb300 import binding as pb  # noqa: E402
from tests import test_block_zero_scales_gpu as zs  # noqa: E402


@pytest.mark.parametrize("rows", [1, 70])
@pytest.mark.parametrize("L", [70, 5000])
@pytest.mark.parametrize("v_scale", [2.0 ** 100, 2.0 ** 115, 2.0 ** 119])
@pytest.mark.parametrize("sinks", [False, True])
def test_the_largest_scales(rows, L, v_scale, sinks):
    got = zs._run(L, rows, pb.CODE_INT8, v_scale, sinks)
    zs._close(got, L, v_scale, pb.CODE_INT8)
