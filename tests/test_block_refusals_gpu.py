"""The binding of the 8-bit serving step refuses tensors of another type, shape or device before it calls the library."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from paged_kv_gqa_12_gb300 import binding as pb  # noqa: E402

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

_k = dict(dtype=torch.int32, device="cuda")


def _refuses(call, base, **bad):
    for name, value in bad.items():
        with pytest.raises((ValueError, pb.PaError)):
            call(**{**base, name: value})
    call(**base)
    torch.cuda.synchronize()


def test_tables():
    z = lambda n: torch.zeros(n, **_k)      # noqa: E731
    base = dict(context_lens=z(3), new_lens=z(3), page_counts=z(3), free_pages=torch.arange(8, **_k),
                free_count=torch.full((1,), 8, **_k), block_table=torch.zeros(3, 4, **_k), page_size=16, num_pages=8,
                seq_lens=z(3), query_start_loc=z(4), slots=torch.zeros(5, dtype=torch.int64, device="cuda"), positions=z(5))

    def call(context_lens, new_lens, page_counts, free_pages, free_count, block_table, **kw):
        pb.step_tables(context_lens, new_lens, page_counts, free_pages, free_count, block_table, **kw)
    _refuses(call, base, context_lens=z(3).cpu(), new_lens=z(2), page_counts=z(3).long(), free_count=z(2),
             block_table=torch.zeros(2, 4, **_k), seq_lens=z(4), query_start_loc=z(3), slots=z(5), positions=z(4),
             page_size=0, free_pages=torch.zeros(8, device="cuda"))
    with pytest.raises(ValueError):
        call(**base, page_counts_out=z(2))
    with pytest.raises(ValueError):
        call(**base, scratch=torch.zeros(10, dtype=torch.uint8, device="cuda"))


def _cache():
    c = lambda dt: torch.zeros(6, 16, 2, 64, dtype=dt, device="cuda")      # noqa: E731
    return c(torch.int8), c(torch.int8), torch.ones(6, 2, device="cuda"), torch.ones(6, 2, device="cuda")


def test_append():
    kc, vc, ks, vs = _cache()
    new = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    base = dict(k_new=new, v_new=new.clone(), k_cache=kc, v_cache=vc, k_scales=ks, v_scales=vs,
                block_table=torch.arange(6, **_k).view(2, 3), seq_lens=torch.tensor([5, 9], **_k),
                query_start_loc=torch.tensor([0, 1, 4], **_k))

    def call(k_new, v_new, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, **kw):
        pb.append_blocks(k_new, v_new, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, **kw)
    _refuses(call, base, k_new=new.float(), v_new=new[:3], k_cache=kc.to(torch.uint8), v_cache=vc[:5], k_scales=ks[:5],
             v_scales=vs.double(), block_table=torch.zeros(1, 3, **_k), seq_lens=torch.zeros(2, device="cuda"),
             query_start_loc=torch.zeros(2, **_k))
    with pytest.raises(ValueError):
        call(**{**base, "k_new": new.cpu(), "v_new": new.cpu()})
    with pytest.raises(pb.PaError):                # one token a request: as many rows as requests
        call(**{**base, "query_start_loc": None})


def test_attend():
    kc, vc, ks, vs = _cache()
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device="cuda")
    plan = pb.block_plan(num_q_heads=4, num_kv_heads=2, head_dim=64, page_size=16, code=pb.CODE_INT8, max_batch=2,
                         max_pages_per_seq=3, max_total_q=4, max_new=3)
    scratch = pb.alloc_scratch(plan)
    base = dict(q=q, k_cache=kc, v_cache=vc, k_scales=ks, v_scales=vs, block_table=torch.arange(6, **_k).view(2, 3),
                seq_lens=torch.tensor([5, 9], **_k), query_start_loc=torch.tensor([0, 1, 4], **_k), scale=0.125,
                out=torch.empty_like(q), lse=torch.empty(4, 4, device="cuda"), scratch=scratch)

    def call(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, **kw):
        pb.block_attend(plan, q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, **kw)
    u8 = kc.view(torch.uint8)
    _refuses(call, base, q=q.half(), k_cache=u8, v_cache=vc[:, :8], k_scales=ks.t().contiguous().t(), v_scales=vs[:5],
             block_table=torch.zeros(2, 2, **_k), seq_lens=torch.zeros(3, **_k), query_start_loc=torch.zeros(4, **_k),
             out=torch.empty(4, 4, 128, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(4, 3, device="cuda"),
             sinks=torch.zeros(4, device="cuda"), scratch=scratch[:1000], scale=float("nan"))
    for name in ("q", "k_scales", "out"):
        with pytest.raises(ValueError):
            call(**{**base, name: base[name].cpu()})
    with pytest.raises(ValueError):
        call(**{**base, "k_cache": u8, "v_cache": vc.view(torch.uint8)})       # e4m3 codes for an int8 plan


def test_verify():
    p = torch.full((4, 10), 0.1, device="cuda")
    base = dict(tokens=torch.zeros(4, **_k), target_probs=p, query_start_loc=torch.tensor([0, 1, 4], **_k),
                accept_u=torch.zeros(4, device="cuda"), sample_u=torch.zeros(2, device="cuda"),
                out_tokens=torch.zeros(2, 4, **_k), num_tokens=torch.zeros(2, **_k), draft_probs=p.clone())

    def call(tokens, target_probs, query_start_loc, accept_u, sample_u, out_tokens, num_tokens, **kw):
        pb.verify_tokens(tokens, target_probs, query_start_loc, accept_u, sample_u, out_tokens, num_tokens, **kw)
    _refuses(call, base, tokens=torch.zeros(3, **_k), target_probs=p.half(), query_start_loc=torch.zeros(4, **_k),
             accept_u=torch.zeros(4, **_k), sample_u=torch.zeros(3, device="cuda"), out_tokens=torch.zeros(3, 4, **_k),
             num_tokens=torch.zeros(2, device="cuda"), draft_probs=p[:3])
    with pytest.raises(ValueError):
        call(**{**base, "target_probs": p.cpu()})
