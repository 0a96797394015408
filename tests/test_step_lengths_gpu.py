"""The lengths that a server carries from step to step: prompts that need one token, drafts that are not accepted, requests
that end, and a step that does not fit, which leaves everything as it was."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from paged_kv_gqa_12_gb300 import binding as pb  # noqa: E402
from tests import block_refs as ref  # noqa: E402

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

_k = dict(dtype=torch.int32, device="cuda")


def test_lengths_of_mixed_and_refused_steps():
    B, W, pool, Hq, Hkv, D, V, most = 5, 8, 14, 8, 2, 64, 200, 40
    g = torch.Generator().manual_seed(11)
    plan = pb.block_plan(num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=16, code=pb.CODE_INT8, max_batch=B,
                         max_pages_per_seq=W, max_total_q=200, max_new=most)
    scratch = pb.alloc_scratch(plan)
    context_lens, page_counts = torch.zeros(B, **_k), torch.zeros(B, **_k)
    free_pages, free_count = torch.arange(pool, **_k), torch.tensor([pool], **_k)
    block_table, seq_lens, qsl = torch.zeros(B, W, **_k), torch.zeros(B, **_k), torch.zeros(B + 1, **_k)
    slots, positions = torch.zeros(200, dtype=torch.int64, device="cuda"), torch.zeros(200, **_k)
    k_cache, v_cache = (torch.zeros(pool, 16, Hkv, D, dtype=torch.int8, device="cuda") for _ in range(2))
    k_scales, v_scales = torch.zeros(pool, Hkv, device="cuda"), torch.zeros(pool, Hkv, device="cuda")
    out_tokens, num_tokens = torch.zeros(B, most, **_k), torch.zeros(B, **_k)
    want = [0] * B
    # (new tokens, rows that need a token) of each request; the third step needs more pages than are free
    steps = [([40, 17, 3, 30, 1], [1, 1, 1, 1, 1]), ([4, 1, 3, 2, 5], [4, 1, 3, 2, 5]), ([40, 40, 40, 1, 1], [1, 1, 1, 1, 1]),
             ([4, -1, 3, 1, 5], [4, 0, 3, 1, 5]), ([2, 40, 1, -1, 3], [2, 1, 1, 0, 3])]
    for step, (new, verify) in enumerate(steps):
        refused = step == 2
        before = block_table.clone(), free_count.clone(), page_counts.clone()
        new_lens, verify_lens = torch.tensor(new, **_k), torch.tensor(verify, **_k)
        pb.step_tables(context_lens, new_lens, page_counts, free_pages, free_count, block_table, page_size=16,
                       num_pages=pool, seq_lens=seq_lens, query_start_loc=qsl, slots=slots, positions=positions,
                       scratch=scratch)
        T = sum(max(n, 0) for n in new)
        k, v = (torch.randn(T, Hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
        q = torch.randn(T, Hq, D, generator=g).bfloat16().cuda()
        out, lse = torch.full_like(q, 7.0), torch.full((T, Hq), 7.0, device="cuda")
        pb.append_blocks(k, v, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, query_start_loc=qsl,
                         scratch=scratch)
        pb.block_attend(plan, q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, query_start_loc=qsl,
                        scale=D ** -0.5, out=out, lse=lse, scratch=scratch)
        rows = torch.minimum(verify_lens, qsl[1:] - qsl[:-1])
        loc = torch.nn.functional.pad(rows.cumsum(0, dtype=torch.int32), (1, 0))
        R = sum(verify)
        p = torch.softmax(2 * torch.randn(R, V, generator=g), -1)
        tokens = torch.randint(0, V, (R,), generator=g).to(torch.int32)
        u, w = 0.01 * torch.rand(R, generator=g), torch.rand(B, generator=g)
        pb.verify_tokens(tokens.cuda(), p.cuda(), loc, u.cuda(), w.cuda(), out_tokens, num_tokens, scratch=scratch)
        context_lens = seq_lens - rows + num_tokens

        assert pb.check(scratch) == (pb.DEVICE_NO_PAGES if refused else 0)
        if refused:
            assert all(torch.equal(a, b) for a, b in zip(before, (block_table, free_count, page_counts)))
            assert (out == 7).all() and (lse == 7).all() and num_tokens.tolist() == [0] * B and (slots == -1).all()
        else:
            h_loc = [0]
            for n in verify:
                h_loc.append(h_loc[-1] + n)
            _, kept = ref.verify(tokens, p, None, h_loc, u, w, most)
            assert num_tokens.tolist() == kept.tolist()
            want = [0 if n < 0 else c + n - r + int(a) for c, n, r, a in zip(want, new, verify, kept)]
            assert (lse != 7).all()
        assert context_lens.tolist() == want, (step, context_lens.tolist(), want)
