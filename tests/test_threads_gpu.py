"""Calls from several host threads."""
import threading

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


def problem(D, n, heads, seed, ps=16):
    """One request of n pages in order: (q, k, v, lens)."""
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(n, ps, 1, D, generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn(1, heads, D, generator=g).bfloat16().cuda()
    return q, k, v, torch.tensor([n * ps - 3], dtype=torch.int32, device="cuda")


def sparse_job(pb, D, top):
    n = 12
    q, k, v, lens = problem(D, n, 4, top)
    plan = pb.sparse_plan(num_q_heads=4, num_kv_heads=1, head_dim=D, page_size=16, max_batch=1, max_pages_per_seq=n,
                          max_total_q=1, top_pages=top, num_splits=1)
    bt = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    pages = torch.full((1, 1, top), -1, dtype=torch.int32, device="cuda")
    pages[0, 0, :n] = bt[0]
    out, scratch = torch.empty_like(q), pb.alloc_scratch(plan)
    return (lambda stream: pb.sparse_attend(plan, q, k, v, bt, lens, pages, scale=0.06, out=out, scratch=scratch,
                                            stream=stream)), [out]


def dense_job(pb, D, width, mode):
    n = 12
    q, k, v, lens = problem(D, n, 4, width)
    plan = pb.plan(mode=mode, num_q_heads=4, num_kv_heads=1, head_dim=D, page_size=16, max_batch=1,
                   max_pages_per_seq=width, num_splits=1, max_total_q=1 if mode == pb.MODE_EXTEND else 0)
    bt = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    bt[0, :n] = torch.arange(n, device="cuda")
    qsl = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    out, scratch = torch.empty_like(q), pb.alloc_scratch(plan)
    if mode == pb.MODE_EXTEND:
        return (lambda stream: pb.extend(plan, q, k, v, bt, lens, qsl, scale=0.125, out=out, scratch=scratch,
                                         stream=stream)), [out]
    return (lambda stream: pb.decode(plan, q, k, v, bt, lens, scale=0.125, out=out, scratch=scratch,
                                     stream=stream)), [out]


def in_threads(calls, times):
    """Each of ``calls`` (stream -> None) ``times`` times in a thread and stream of its own; returns the errors."""
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(len(calls))

    def work(call, stream):
        start.wait()
        for _ in range(times):
            try:
                call(stream)
            except Exception as e:          # noqa: BLE001 (the test reports whatever came)
                errors.append(repr(e))
                return
    threads = [threading.Thread(target=work, args=x) for x in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


def check(jobs, times):
    """jobs: [(call, outputs)].  First alone, then each in a thread: no error, the same outputs."""
    want = []
    for call, outs in jobs:
        call(torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append([x.clone() for x in outs])
        for x in outs:
            x.zero_()
    assert in_threads([call for call, _ in jobs], times) == []
    for (_, outs), ref in zip(jobs, want):
        for x, y in zip(outs, ref):
            assert torch.equal(x, y)


@pytest.mark.parametrize("kind", ["sparse", "decode", "extend"])
def test_first_cuda_call_of_a_thread(pb, kind):
    # the thread has made no other CUDA call: nothing has made a context current in it
    check([sparse_job(pb, 128, 16) if kind == "sparse" else
           dense_job(pb, 128, 100, pb.MODE_DECODE if kind == "decode" else pb.MODE_EXTEND)], 1)
