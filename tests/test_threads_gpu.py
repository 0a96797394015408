"""Calls from several host threads."""
import ctypes
import os
import shutil
import subprocess
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


# Plans of one kernel whose shared memory differs, from two host threads in C (no
# interpreter between their calls): each call has to be launched with its own size.

HAMMER = r"""
#include <pthread.h>
#include "pa.h"

typedef struct {
  int32_t kind, times;
  const void *plan, *q, *k, *v, *pages, *bt, *lens;
  void *out, *scratch, *stream;
  int64_t bytes, heads, dim, n;
  int32_t width, status;
} job;

static void* work(void* x) {
  job* j = x;
  const int64_t row = j->heads * j->dim, ps = 16, d = j->dim;
  for (int i = 0; i < j->times && j->status == PA_OK; ++i) {
    if (j->kind == 0)
      j->status = pa_decode(j->plan, j->q, row, d, j->k, j->v, ps * d, d, d, j->n, j->bt, j->width, j->lens, 1, 0.1f,
                            NULL, 1.f, 1.f, NULL, NULL, j->out, row, d, NULL, j->scratch, j->bytes, j->stream);
    else if (j->kind == 1)
      j->status = pa_sparse_attend(j->plan, j->q, row, d, j->k, j->v, ps * d, d, d, j->n, j->bt, j->width, j->lens, NULL,
                                   1, 1, j->pages, 0.1f, NULL, 1.f, 1.f, NULL, NULL, j->out, row, d, NULL, j->scratch,
                                   j->bytes, j->stream);
    else
      j->status = pa_select_pages(j->plan, j->q, row, d, j->k, 2 * d, 2 * d, j->n, j->bt, j->width, j->lens, NULL, 1, 1,
                                  j->out, j->scratch, j->bytes, j->stream);
  }
  return NULL;
}

int hammer(job* jobs, int n) {
  pthread_t t[8];
  if (n > 8) return 1;
  for (int i = 0; i < n; ++i)
    if (pthread_create(&t[i], NULL, work, &jobs[i])) return 1;
  for (int i = 0; i < n; ++i) pthread_join(t[i], NULL);
  return 0;
}
"""


class Job(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("kind", "times")] +
                [(n, ctypes.c_void_p) for n in ("plan", "q", "k", "v", "pages", "bt", "lens", "out", "scratch", "stream")] +
                [(n, ctypes.c_int64) for n in ("bytes", "heads", "dim", "n")] +
                [(n, ctypes.c_int32) for n in ("width", "status")])


@pytest.fixture(scope="module")
def hammer(pb, tmp_path_factory):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    from paged_kv_gqa_12_gb300 import build
    src = tmp_path_factory.mktemp("hammer") / "hammer.c"
    src.write_text(HAMMER)
    so = src.with_suffix(".so")
    r = subprocess.run([cc, "-std=c11", "-O1", "-shared", "-fPIC", "-pthread", "-I" + build.INCLUDE, str(src),
                        build.LIB_PATH, "-Wl,-rpath," + os.path.dirname(build.LIB_PATH), "-o", str(so)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(str(so))


@pytest.mark.parametrize("kind", ["decode", "sparse", "select"])
def test_two_plans_of_one_kernel(pb, hammer, kind):
    keep, jobs = [], []
    # decode: block-table entries held by a CTA; sparse: entries of a page list; select: heads of a group
    for i, size in enumerate({"decode": (30000, 100), "sparse": (4096, 64), "select": (128, 64)}[kind]):
        D, n, heads = (64, 12, 4) if kind == "decode" else (256, 12, 4) if kind == "sparse" else (256, 40, size)
        q, k, v, lens = problem(D, n, heads, size)
        width, out, pages = n, torch.zeros_like(q), None
        if kind == "decode":
            width = size
            plan = pb.plan(mode=pb.MODE_DECODE, num_q_heads=heads, num_kv_heads=1, head_dim=D, page_size=16, max_batch=1,
                           max_pages_per_seq=width, num_splits=1)
        else:
            top = size if kind == "sparse" else 8
            plan = pb.sparse_plan(num_q_heads=heads, num_kv_heads=1, head_dim=D, page_size=16, max_batch=1,
                                  max_pages_per_seq=n, max_total_q=1, top_pages=top, num_splits=1)
        if kind == "sparse":
            pages = torch.full((1, 1, size), -1, dtype=torch.int32, device="cuda")
            pages[0, 0, :n] = torch.arange(n, device="cuda")
        if kind == "select":
            k = torch.stack([k.amin(1), k.amax(1)], 2)
            out = torch.zeros(1, 1, 8, dtype=torch.int32, device="cuda")
        bt = torch.zeros(1, width, dtype=torch.int32, device="cuda")
        bt[0, :n] = torch.arange(n, device="cuda")
        scratch, stream = pb.alloc_scratch(plan), torch.cuda.Stream()
        jobs.append(Job(kind=("decode", "sparse", "select").index(kind), times=1, plan=ctypes.addressof(plan),
                        q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), pages=None if pages is None else pages.data_ptr(),
                        bt=bt.data_ptr(), lens=lens.data_ptr(), out=out.data_ptr(), scratch=scratch.data_ptr(),
                        stream=stream.cuda_stream, bytes=scratch.nbytes, heads=heads, dim=D, n=n, width=width))
        keep.append((plan, q, k, v, lens, pages, bt, scratch, stream, out))
    torch.cuda.synchronize()
    array = (Job * len(jobs))(*jobs)
    want = []
    for i in range(len(jobs)):                            # one thread at a time
        assert hammer.hammer(ctypes.byref(array, i * ctypes.sizeof(Job)), 1) == 0 and array[i].status == 0
        torch.cuda.synchronize()
        want.append(keep[i][-1].clone())
        keep[i][-1].zero_()
        array[i].times = 4000
    torch.cuda.synchronize()
    assert hammer.hammer(array, len(jobs)) == 0
    torch.cuda.synchronize()
    assert [pb.status_string(j.status) for j in array] == [pb.status_string(0)] * len(jobs)
    for x, y in zip(keep, want):
        assert torch.equal(x[-1], y) and y.any()
