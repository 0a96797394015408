"""Tensors that the long-context calls turn down in the binding, before anything is
enqueued: workspaces and rotation tables of another device, kind or size."""
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


def calls(pb):
    """The four calls on one small request, as functions of their workspace."""
    D, ps, n = 64, 16, 4
    dev = "cuda"
    bf = dict(dtype=torch.bfloat16, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    kc, vc = torch.zeros(n, ps, 1, D, **bf), torch.zeros(n, ps, 1, D, **bf)
    new, q = torch.ones(1, 1, D, **bf), torch.ones(1, 4, D, **bf)
    bounds, bt, lens = torch.zeros(n, 1, 2, D, **bf), torch.arange(n, **i32)[None], torch.tensor([n * ps], **i32)
    pages = torch.arange(2, **i32)[None, None].contiguous()
    rope = pb.rope(torch.ones(8, D, device=dev), rot_dim=D)
    pos, slots = torch.zeros(1, **i32), torch.zeros(1, dtype=torch.int64, device=dev)
    plan = pb.sparse_plan(num_q_heads=4, num_kv_heads=1, head_dim=D, page_size=ps, max_batch=1, max_pages_per_seq=n,
                          max_total_q=1, top_pages=2, last_pages=1)
    return rope, plan, {
        "append": lambda s: pb.append_rope_kv(rope, new, new, pos, kc, vc, slots, scratch=s),
        "bounds": lambda s: pb.page_bounds(kc, bt, lens, bounds, scratch=s),
        "select": lambda s: pb.select_pages(plan, q, bounds, bt, lens, pages, scratch=s),
        "attend": lambda s: pb.sparse_attend(plan, q, kc, vc, bt, lens, pages, scale=1.0, out=torch.empty_like(q),
                                             scratch=s)}


@pytest.mark.parametrize("name", ["append", "bounds", "select", "attend"])
def test_workspaces(pb, name):
    _, plan, fs = calls(pb)
    f = fs[name]
    good = pb.alloc_scratch(plan)
    f(good)
    assert pb.check(good) == 0
    n = good.numel()
    for bad in (torch.zeros(n, dtype=torch.uint8), torch.zeros(n, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(ValueError, match="scratch"):
            f(bad)
    if name in ("append", "bounds"):
        with pytest.raises(ValueError, match="header"):
            f(good[:1024])
        f(None)
    else:
        with pytest.raises(pb.PaError) as e:
            f(good[:1024])
        assert e.value.status == pb.PA_ERR_SCRATCH_TOO_SMALL
    wide = torch.zeros(n + 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(pb.PaError) as e:
        f(wide[1:n + 1])                          # not aligned to the error word
    assert e.value.status == pb.PA_ERR_UNSUPPORTED
    torch.cuda.synchronize()


def test_rotation_tables_of_another_device(pb):
    rope, _, fs = calls(pb)
    assert rope.device == torch.cuda.current_device()
    fs["append"](None)
    rope.device += 1                              # as if another device had been current when it was made
    with pytest.raises(ValueError, match="device"):
        fs["append"](None)
    torch.cuda.synchronize()
