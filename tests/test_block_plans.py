"""Plans of pa_block_attend for decode: one row a request can always be asked for without query_start_loc."""
import pytest

from paged_kv_gqa_12_gb300 import binding as pb
from paged_kv_gqa_12_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


@pytest.mark.parametrize("group", [1, 8, 16, 48, 49, 64, 71, 128])
@pytest.mark.parametrize("kv_heads,batch", [(1, 1), (1, 303), (1, 304), (1, 4096), (8, 64), (2, 65535)])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_decode_plans_are_not_chunked(group, kv_heads, batch, head_dim):
    p = pb.block_plan(num_q_heads=group * kv_heads, num_kv_heads=kv_heads, head_dim=head_dim, page_size=16, code=pb.CODE_INT8,
                      max_batch=batch, max_pages_per_seq=512, max_total_q=batch, max_new=1, num_sms=152)
    assert p.chunked == 0 and p.row_groups == -(-group // (8 if group <= 8 else 16))
