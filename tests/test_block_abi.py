"""The calls of the 8-bit serving step on the host: plans, refusals before anything is enqueued, the C header."""
import ctypes
import os
import shutil
import subprocess

import pytest

from paged_kv_gqa_12_gb300 import binding as pb
from paged_kv_gqa_12_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, SMALL = pb.PA_OK, pb.PA_ERR_INVALID_ARG, pb.PA_ERR_UNSUPPORTED, pb.PA_ERR_SCRATCH_TOO_SMALL
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pb.load()


def _plan(**kw):
    a = dict(num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16, code=pb.CODE_INT8, max_batch=64,
             max_pages_per_seq=512, max_total_q=256, max_new=4, num_sms=152)
    a.update(kw)
    return pb.block_plan(**a)


@pytest.mark.parametrize("bad,status", [
    (dict(code=2), INVALID), (dict(code=-1), INVALID), (dict(max_new=0), INVALID), (dict(num_q_heads=30), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(num_q_heads=129 * 8), UNSUPPORTED),
    (dict(window=-1), INVALID), (dict(soft_cap=-1.0), INVALID), (dict(soft_cap=float("nan")), INVALID),
    (dict(max_batch=-1), INVALID), (dict(max_batch=65536), UNSUPPORTED), (dict(max_total_q=-1), INVALID),
    (dict(max_pages_per_seq=1 << 27), UNSUPPORTED), (dict(num_ctas=-1), INVALID),
    (dict(host_seq_lens=[5, -1]), INVALID), (dict(host_seq_lens=[512 * 16 + 1]), INVALID),
    (dict(host_seq_lens=[1] * 65), INVALID),
])
def test_plan_rejects(lib, bad, status):
    with pytest.raises(pb.PaError) as e:
        _plan(**bad)
    assert e.value.status == status


def test_plans(lib):
    p = _plan()
    assert p.chunked == 0 and p.row_groups == 1 and p.ctas >= 152 and p.smem_bytes <= 232448
    rows = 2 * p.ctas * p.head_group * 16                 # two parts a CTA, 16 rows a head
    assert p.scratch_bytes == pb.SCRATCH_HEADER_BYTES + rows * 128 * 4 + rows * 4 + 32 * p.ctas
    assert _plan(max_new=1, max_total_q=64).row_groups == 1
    assert _plan(max_new=12).row_groups == 3 and _plan(max_new=12).chunked == 0
    c = _plan(max_new=13)
    assert c.chunked == 1 and 1 <= c.group_requests <= 64
    # requests too few to fill the card in chunks: up to 128 rows a kv head are split
    assert _plan(max_new=32, max_batch=4).row_groups == 8 and _plan(max_new=33, max_batch=4).chunked == 1
    # a copy of at most 2 GiB, or of one request
    assert c.group_requests * 512 * 16 * 8 * 128 * 4 <= 1 << 31
    one = _plan(max_new=100, max_pages_per_seq=1 << 17)
    assert one.group_requests == 1
    # short contexts do not need a whole wave of CTAs; the lengths may say so
    assert _plan(max_batch=1, max_pages_per_seq=8, max_total_q=1, max_new=1).ctas <= 8
    assert _plan(host_seq_lens=[100] * 4).ctas < _plan(host_seq_lens=[8000] * 64).ctas == p.ctas
    assert _plan(num_ctas=5).ctas == 5
    # a CTA takes as many heads as divide Hkv, up to its warps, and then as many more keys
    def heads(h, batch=64):
        q = _plan(num_kv_heads=h, num_q_heads=h, max_new=1, max_batch=batch)
        return q.head_group, q.tile_tokens * q.head_group
    assert [heads(h)[0] for h in (1, 2, 3, 4, 6, 8)] == [1, 2, 1, 4, 2, 4] and heads(8, 1)[0] == 4
    assert len({heads(h)[1] for h in (1, 2, 3, 8)}) == 1
    assert _plan(max_batch=0, max_total_q=0, max_pages_per_seq=0).ctas == 1


def test_plan_uses_host_lengths(lib):
    a, b = _plan(host_seq_lens=[600] * 64), _plan(host_seq_lens=[8000] * 64)
    assert b.ctas >= a.ctas and a.scratch_bytes <= b.scratch_bytes


def _attend(lib, plan, **over):
    a = dict(q=0x10000, qs=(32 * 128, 128), k=0x20000, v=0x40000, kvs=(16 * 8 * 128, 8 * 128, 128), pages=100,
             ks=0x80000, vs=0x90000, ss=8, bt=0x50000, bts=512, sl=0x60000, qsl=0x68000, batch=4, T=9, scale=0.088,
             sinks=None, out=0x70000, os=(32 * 128, 128), lse=None, scratch=0x100000, bytes=plan.scratch_bytes)
    a.update(over)
    return lib.pa_block_attend(ctypes.byref(plan), vp(a["q"]), *a["qs"], vp(a["k"]), vp(a["v"]), *a["kvs"], a["pages"],
                               vp(a["ks"]), vp(a["vs"]), a["ss"], vp(a["bt"]), a["bts"], vp(a["sl"]), vp(a["qsl"]),
                               a["batch"], a["T"], a["scale"], vp(a["sinks"]), vp(a["out"]), *a["os"], vp(a["lse"]),
                               vp(a["scratch"]), a["bytes"], None)


@pytest.mark.parametrize("over,status", [
    (dict(batch=65), INVALID), (dict(batch=-1), INVALID), (dict(T=257), INVALID), (dict(T=-1), INVALID),
    (dict(qsl=None), INVALID),                             # one row a request needs as many rows as requests
    (dict(scale=float("inf")), INVALID), (dict(sinks=0x1000), INVALID), (dict(scratch=None), INVALID),
    (dict(bytes=65535), SMALL), (dict(scratch=0x100080), UNSUPPORTED), (dict(q=None), INVALID), (dict(q=0x10002), UNSUPPORTED),
    (dict(out=None), INVALID), (dict(out=0x70002), UNSUPPORTED), (dict(qs=(32 * 128 + 1, 128)), UNSUPPORTED),
    (dict(qs=(0, 128)), INVALID), (dict(os=(32 * 128, -128)), INVALID), (dict(k=None), INVALID), (dict(k=0x20008), UNSUPPORTED),
    (dict(kvs=(16 * 8 * 128, 8 * 128 + 8, 128)), UNSUPPORTED), (dict(kvs=(0, 8 * 128, 128)), INVALID), (dict(pages=0), INVALID),
    (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(ks=0x80002), UNSUPPORTED), (dict(ss=7), INVALID),
    (dict(ss=-1), INVALID), (dict(bt=None), INVALID), (dict(sl=None), INVALID), (dict(bts=-1), INVALID),
    (dict(lse=0x1001), UNSUPPORTED), (dict(sl=0x60002), UNSUPPORTED),
    (dict(batch=0), OK), (dict(T=0, batch=0, qsl=None), OK), (dict(T=0), OK),
])
def test_attend_rejects_before_launch(lib, over, status):
    assert _attend(lib, _plan(), **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(q=0x10008), UNSUPPORTED), (dict(out=0x70008), UNSUPPORTED), (dict(qs=(32 * 128 + 4, 128)), UNSUPPORTED),
    (dict(os=(32 * 128, 132)), UNSUPPORTED), (dict(qsl=None, T=4), INVALID)])
def test_chunked_attend_rejects_before_launch(lib, over, status):
    assert _attend(lib, _plan(max_new=100), **over) == status


def test_attend_rejects_hand_edited_plans(lib):
    for plan, edits in ((_plan(), dict(chunked=1)), (_plan(max_new=100), dict(chunked=0)), (_plan(), dict(ctas=0)),
                        (_plan(), dict(row_groups=2)), (_plan(), dict(tile_tokens=8)), (_plan(), dict(head_group=1)),
                        (_plan(), dict(smem_bytes=1000)), (_plan(), dict(min_tiles=0)),
                        (_plan(), dict(ctas=20000)), (_plan(), dict(ctas=10000)),
                        (_plan(max_new=100), dict(group_requests=0)), (_plan(max_new=100), dict(group_requests=60000))):
        for k, v in edits.items():
            setattr(plan, k, v)
        assert _attend(lib, plan, bytes=1 << 40) == INVALID, edits
    plan = _plan()
    plan.shape.code = 5
    assert _attend(lib, plan) == INVALID


def _append(lib, **over):
    a = dict(k=0x10000, v=0x20000, ns=(8 * 128, 128), kc=0x30000, vc=0x40000, kvs=(16 * 8 * 128, 8 * 128, 128), pages=100,
             ps=16, H=8, D=128, code=1, ks=0x50000, vs=0x60000, ss=8, bt=0x70000, bts=64, W=64, sl=0x80000, qsl=0x90000,
             batch=4, T=9, scratch=None)
    a.update(over)
    return lib.pa_append_blocks(vp(a["k"]), vp(a["v"]), *a["ns"], vp(a["kc"]), vp(a["vc"]), *a["kvs"], a["pages"], a["ps"],
                                a["H"], a["D"], a["code"], vp(a["ks"]), vp(a["vs"]), a["ss"], vp(a["bt"]), a["bts"],
                                a["W"], vp(a["sl"]), vp(a["qsl"]), a["batch"], a["T"], vp(a["scratch"]), None)


@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(pages=0), INVALID), (dict(W=-1), INVALID),
    (dict(code=2), INVALID), (dict(D=96), UNSUPPORTED), (dict(ps=8), UNSUPPORTED), (dict(qsl=None), INVALID),
    (dict(k=None), INVALID), (dict(k=0x10008), UNSUPPORTED), (dict(ns=(8 * 128 + 4, 128)), UNSUPPORTED),
    (dict(ns=(0, 128)), INVALID), (dict(kc=0x30008), UNSUPPORTED), (dict(kvs=(16 * 8 * 128, 8 * 128, 120)), UNSUPPORTED),
    (dict(kvs=(-1, 8 * 128, 128)), INVALID), (dict(ks=None), INVALID), (dict(vs=0x60001), UNSUPPORTED), (dict(ss=4), INVALID),
    (dict(bt=None), INVALID), (dict(bts=63), INVALID), (dict(sl=None), INVALID), (dict(W=1 << 27, bts=1 << 27), UNSUPPORTED),
    (dict(T=1 << 30, H=64, ss=64), UNSUPPORTED), (dict(scratch=0x101), UNSUPPORTED),
    (dict(batch=0), OK), (dict(T=0), OK),
])
def test_append_rejects_before_launch(lib, over, status):
    assert _append(lib, **over) == status


def _tables(lib, **over):
    a = dict(ctx=0x1000, new=0x2000, B=4, ps=16, held=0x3000, held_out=0x3000, free=0x4000, cap=100, count=0x5000,
             count_out=0x5000, pages=100, bt=0x6000, bts=32, W=32, sl=0x7000, qsl=0x8000, slots=0x9000, pos=0xa000, T=64,
             scratch=None)
    a.update(over)
    return lib.pa_step_tables(vp(a["ctx"]), vp(a["new"]), a["B"], a["ps"], vp(a["held"]), vp(a["held_out"]), vp(a["free"]),
                              a["cap"], vp(a["count"]), vp(a["count_out"]), a["pages"], vp(a["bt"]), a["bts"], a["W"],
                              vp(a["sl"]), vp(a["qsl"]), vp(a["slots"]), vp(a["pos"]), a["T"], vp(a["scratch"]), None)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), INVALID), (dict(B=8193), UNSUPPORTED), (dict(ps=0), INVALID), (dict(cap=-1), INVALID), (dict(pages=0), INVALID),
    (dict(W=-1), INVALID), (dict(T=-1), INVALID), (dict(T=(1 << 29) + 1), UNSUPPORTED), (dict(cap=(1 << 30) + 1), UNSUPPORTED),
    (dict(W=1 << 27, bts=1 << 27), UNSUPPORTED), (dict(ctx=None), INVALID), (dict(new=None), INVALID),
    (dict(held=None), INVALID), (dict(held_out=None), INVALID), (dict(free=None), INVALID), (dict(count=None), INVALID),
    (dict(count_out=None), INVALID), (dict(bt=None), INVALID), (dict(bts=31), INVALID), (dict(sl=None), INVALID),
    (dict(qsl=None), INVALID), (dict(slots=None), INVALID), (dict(pos=None), INVALID), (dict(slots=0x9004), UNSUPPORTED),
    (dict(ctx=0x1002), UNSUPPORTED), (dict(scratch=0x1002), UNSUPPORTED),
])
def test_tables_reject_before_launch(lib, over, status):
    assert _tables(lib, **over) == status


def _verify(lib, **over):
    a = dict(tok=0x1000, p=0x2000, ps=1000, q=0x3000, qs=1000, V=1000, qsl=0x4000, B=4, T=9, u=0x5000, w=0x6000, out=0x7000,
             os=8, W=8, num=0x8000, scratch=None)
    a.update(over)
    return lib.pa_verify_tokens(vp(a["tok"]), vp(a["p"]), a["ps"], vp(a["q"]), a["qs"], a["V"], vp(a["qsl"]), a["B"], a["T"],
                                vp(a["u"]), vp(a["w"]), vp(a["out"]), a["os"], a["W"], vp(a["num"]), vp(a["scratch"]), None)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(V=0), INVALID), (dict(W=-1), INVALID), (dict(V=(1 << 20) + 1), UNSUPPORTED),
    (dict(tok=None), INVALID), (dict(p=None), INVALID), (dict(ps=999), INVALID), (dict(qs=999), INVALID), (dict(qsl=None), INVALID),
    (dict(u=None), INVALID), (dict(w=None), INVALID), (dict(out=None), INVALID), (dict(os=7), INVALID), (dict(num=None), INVALID),
    (dict(p=0x2002), UNSUPPORTED), (dict(num=0x8001), UNSUPPORTED), (dict(B=0), OK),
])
def test_verify_rejects_before_launch(lib, over, status):
    assert _verify(lib, **over) == status


SOURCE = r"""
#include "pa.h"
int main(void) {
  pa_block_shape s = {0};
  s.num_q_heads = 32; s.num_kv_heads = 8; s.head_dim = 128; s.page_size = 16; s.code = PA_CODE_INT8;
  s.max_batch = 4; s.max_pages_per_seq = 8; s.max_total_q = 16; s.max_new = 4; s.num_sms = 152;
  pa_block_plan_t plan;
  const int32_t lens[4] = {1, 2, 3, 4};
  pa_status st = pa_block_plan(&s, lens, 4, &plan);
  if (st != PA_OK) return 1;
  float sc[1] = {0};
  /* nothing to do: every call returns before it touches a pointer or the device */
  st = pa_block_attend(&plan, 0, 0, 0, 0, 0, 0, 0, 0, 0, sc, sc, 0, 0, 0, 0, 0, 0, 0, 1.f, 0, 0, 0, 0, 0,
                       (void*)256, plan.scratch_bytes, 0);
  if (st != PA_OK) return 2;
  st = pa_append_blocks(0, 0, 0, 0, 0, 0, 0, 0, 0, 1, 16, 8, 128, PA_CODE_E4M3, sc, sc, 8, 0, 0, 8, 0, 0, 0, 0, 0, 0);
  if (st != PA_OK) return 3;
  st = pa_verify_tokens(0, 0, 0, 0, 0, 100, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0);
  if (st != PA_OK) return 4;
  st = pa_step_tables(0, 0, -1, 16, 0, 0, 0, 0, 0, 0, 1, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0);
  return st == PA_ERR_INVALID_ARG && PA_DEVICE_NO_PAGES == 32 ? 0 : 5;
}
"""


def test_header_from_c(lib, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "blocks.c"
    src.write_text(SOURCE)
    exe = tmp_path / "blocks"
    subprocess.run([cc, "-std=c11", "-Wall", "-Wextra", "-Werror", "-I" + os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe), build.LIB_PATH, "-Wl,-rpath," + build.OUT_DIR], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
