"""Refusals and planning of the long-context calls, without a GPU: every bad
argument is turned down before anything is enqueued."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from paged_kv_gqa_12_gb300 import binding as pb
from paged_kv_gqa_12_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, SMALL = pb.PA_OK, pb.PA_ERR_INVALID_ARG, pb.PA_ERR_UNSUPPORTED, pb.PA_ERR_SCRATCH_TOO_SMALL
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pb.load()


def ptr(x):
    return vp(x) if x else None


def rope_args(lib, **over):
    r = pb.PaRope(rot_dim=128, interleaved=0, num_axes=1, sections=(ctypes.c_int32 * 4)(64, 0, 0, 0), max_position=100,
                  cos_sin=0x10000, cos_sin_stride=128, q_norm=0x20000, k_norm=0x20100, norm_eps=1e-6, norm_offset=0.0)
    a = dict(q=0x30000, qs=(4096, 128), qo=0x40000, qos=(4096, 128), hq=32, k=0x50000, v=0x60000, ns=(1024, 128),
             pos=0x70000, ps=10, kc=0x80000, vc=0x90000, kvs=(16384, 1024, 128), pages=8, page=16, hkv=8, d=128, kv=0,
             slots=0xa0000, tokens=10, scales=(1.0, 1.0), rope=r)
    for k, v in over.items():
        if hasattr(r, k) and k not in a:
            setattr(r, k, v)
        else:
            a[k] = v
    return lib.pa_append_rope_kv(
        ctypes.byref(a["rope"]) if a["rope"] is not None else None, ptr(a["q"]), *a["qs"], ptr(a["qo"]), *a["qos"],
        a["hq"], ptr(a["k"]), ptr(a["v"]), *a["ns"], ptr(a["pos"]), a["ps"], ptr(a["kc"]), ptr(a["vc"]), *a["kvs"],
        a["pages"], a["page"], a["hkv"], a["d"], a["kv"], ptr(a["slots"]), a["tokens"], *a["scales"], None, None)


@pytest.mark.parametrize("over,status", [
    (dict(rope=None), INVALID), (dict(tokens=-1), INVALID), (dict(tokens=0), OK), (dict(hkv=0), INVALID),
    (dict(pages=0), INVALID), (dict(page=0), INVALID), (dict(kv=2), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(q=0), INVALID), (dict(qo=0), INVALID), (dict(q=0, qo=0), INVALID), (dict(hq=0), INVALID), (dict(hq=-1), INVALID),
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(kc=0), INVALID), (dict(vc=0), INVALID), (dict(slots=0), INVALID),
    (dict(pos=0), INVALID), (dict(cos_sin=None), INVALID), (dict(cos_sin_stride=127), INVALID),
    (dict(cos_sin_stride=130), UNSUPPORTED), (dict(cos_sin=0x10004), UNSUPPORTED), (dict(pos=0x70002), UNSUPPORTED),
    (dict(rot_dim=-8), INVALID), (dict(rot_dim=136), INVALID), (dict(rot_dim=124), UNSUPPORTED),
    (dict(interleaved=2), INVALID), (dict(num_axes=0), INVALID), (dict(num_axes=5), INVALID),
    (dict(num_axes=2), INVALID),                                              # 64 + 0 pairs, but positions of one axis:
    (dict(max_position=0), INVALID), (dict(norm_eps=-1.0), INVALID), (dict(norm_eps=float("nan")), INVALID),
    (dict(norm_offset=float("inf")), INVALID), (dict(q_norm=0x20002), UNSUPPORTED), (dict(k_norm=0x20004), UNSUPPORTED),
    (dict(q=0x30004), UNSUPPORTED), (dict(qos=(4096, 130)), UNSUPPORTED), (dict(ns=(1022, 128)), UNSUPPORTED),
    (dict(ns=(0, 128)), INVALID), (dict(qs=(4096, -128)), INVALID), (dict(kvs=(16384, 1024, 0)), INVALID),
    (dict(kvs=(16384, 1020, 128)), UNSUPPORTED), (dict(kc=0x80008), UNSUPPORTED), (dict(slots=0xa0004), UNSUPPORTED),
    (dict(kv=1, scales=(0.0, 1.0)), INVALID), (dict(kv=1, scales=(1.0, float("nan"))), INVALID),
])
def test_append_rope_refusals(lib, over, status):
    if over == dict(num_axes=2):
        over = dict(num_axes=2, ps=9)
    assert rope_args(lib, **over) == status


def test_append_rope_sections_have_to_sum_up(lib):
    for sec, status in (((16, 24, 23, 0), INVALID), ((16, 24, -1, 0), INVALID)):
        assert rope_args(lib, num_axes=3, sections=(ctypes.c_int32 * 4)(*sec)) == status


def test_sections_of_one_axis(lib):
    sec = lambda *x: (ctypes.c_int32 * 4)(*x)
    for s in (sec(32), sec(63), sec(65), sec(-64)):
        assert rope_args(lib, sections=s) == INVALID
    for s in (sec(64), sec(0), sec(64, 7, 7, 7)):        # all pairs; 0 stands for all
        assert rope_args(lib, sections=s, tokens=0) == OK
    for s in ((16,), (), (33,), (-32, 64), (16, 17)):
        with pytest.raises(ValueError, match="sections|axes"):
            pb.rope(torch.zeros(4, 64), rot_dim=64, sections=s)


def bounds_args(lib, **over):
    a = dict(k=0x10000, kvs=(16384, 1024, 128), pages=8, page=16, hkv=8, d=128, kv=0, bt=0x20000, bts=10, width=10,
             lens=0x30000, qsl=0, batch=4, scale=1.0, scales=0, bounds=0x40000, bs=(2048, 256))
    a.update(over)
    return lib.pa_page_bounds(ptr(a["k"]), *a["kvs"], a["pages"], a["page"], a["hkv"], a["d"], a["kv"], ptr(a["bt"]),
                              a["bts"], a["width"], ptr(a["lens"]), ptr(a["qsl"]), a["batch"], a["scale"],
                              ptr(a["scales"]), ptr(a["bounds"]), *a["bs"], None, None)


@pytest.mark.parametrize("over,status", [
    (dict(batch=0), OK), (dict(batch=-1), INVALID), (dict(k=0), INVALID), (dict(bt=0), INVALID), (dict(lens=0), INVALID),
    (dict(bounds=0), INVALID), (dict(pages=0), INVALID), (dict(hkv=0), INVALID), (dict(kv=3), INVALID),
    (dict(d=80), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(width=11), INVALID),
    (dict(width=-1), INVALID), (dict(kvs=(16384, 0, 128)), INVALID), (dict(kvs=(16384, 1024, 100)), UNSUPPORTED),
    (dict(k=0x10008), UNSUPPORTED), (dict(bounds=0x40008), UNSUPPORTED), (dict(bs=(2044, 256)), UNSUPPORTED),
    (dict(bs=(2048, 0)), INVALID), (dict(kv=1, scale=float("inf")), INVALID),
    (dict(bts=1 << 23, width=1 << 23, batch=256), UNSUPPORTED), (dict(bts=1 << 27, width=1 << 27), UNSUPPORTED),
])
def test_page_bounds_refusals(lib, over, status):
    assert bounds_args(lib, **over) == status


def plan(**over):
    a = dict(num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16, max_batch=64, max_pages_per_seq=2048,
             max_total_q=64, top_pages=128, first_pages=1, last_pages=2, num_sms=152)
    a.update(over)
    return pb.sparse_plan(**a)


@pytest.mark.parametrize("over,status", [
    (dict(num_q_heads=30), INVALID), (dict(num_kv_heads=0), INVALID), (dict(max_batch=-1), INVALID),
    (dict(max_total_q=-1), INVALID), (dict(top_pages=0), INVALID), (dict(last_pages=0), INVALID),
    (dict(first_pages=-1), INVALID), (dict(first_pages=127, last_pages=2), INVALID), (dict(kv_dtype=2), INVALID),
    (dict(soft_cap=-1.0), INVALID), (dict(soft_cap=float("nan")), INVALID), (dict(num_splits=-1), INVALID),
    (dict(head_dim=32), UNSUPPORTED), (dict(page_size=128), UNSUPPORTED), (dict(num_q_heads=129 * 8), UNSUPPORTED),
    (dict(max_pages_per_seq=65537), UNSUPPORTED), (dict(top_pages=4097), UNSUPPORTED),
    (dict(max_total_q=(1 << 24) + 1), UNSUPPORTED),
])
def test_plan_refusals(lib, over, status):
    with pytest.raises(pb.PaError) as e:
        plan(**over)
    assert e.value.status == status


@pytest.mark.parametrize("over", [
    {}, dict(max_total_q=1), dict(max_total_q=20000), dict(num_splits=5), dict(top_pages=4096, last_pages=4000),
    dict(head_dim=256, page_size=64, top_pages=4096), dict(max_pages_per_seq=65536, max_total_q=4096),
    dict(num_q_heads=128, num_kv_heads=1), dict(head_dim=64, page_size=64, kv_dtype=1), dict(max_total_q=0, max_batch=0)])
def test_plan_is_self_consistent(lib, over):
    p = plan(**over)
    # (the kernel's stages are 16, 32 or, for e4m3 keys of 64, 64 keys: whole pages, or pages cut evenly)
    assert p.smem_bytes <= 232448 and p.tile_tokens in (16, 32, 64) and p.score_rows >= 1
    assert p.scratch_bytes >= pb.SCRATCH_HEADER_BYTES
    s = p.shape
    # room for the scores of score_rows rows, and at most about 256 MiB of them
    row = s.num_kv_heads * s.max_pages_per_seq * 4
    assert p.scratch_bytes - pb.SCRATCH_HEADER_BYTES >= p.score_rows * row
    assert p.score_rows == 1 or p.score_rows * row <= 1 << 28
    assert p.scratch_bytes >= pb.SCRATCH_HEADER_BYTES + p.partial_rows * s.num_q_heads * (s.head_dim + 1) * 4


def select_args(lib, p, **over):
    a = dict(q=0x10000, qs=(4096, 128), bounds=0x20000, bs=(2048, 256), pages=100, bt=0x30000, bts=2048, lens=0x40000,
             qsl=0, batch=8, rows=8, out=0x50000, scratch=0x100000, bytes=None)
    a.update(over)
    return lib.pa_select_pages(ctypes.byref(p) if p is not None else None, ptr(a["q"]), *a["qs"], ptr(a["bounds"]),
                               *a["bs"], a["pages"], ptr(a["bt"]), a["bts"], ptr(a["lens"]), ptr(a["qsl"]), a["batch"],
                               a["rows"], ptr(a["out"]), ptr(a["scratch"]),
                               (p.scratch_bytes if p is not None else 0) if a["bytes"] is None else a["bytes"], None)


def attend_args(lib, p, **over):
    a = dict(q=0x10000, qs=(4096, 128), k=0x20000, v=0x28000, kvs=(16384, 1024, 128), pages=100, bt=0x30000, bts=2048,
             lens=0x40000, qsl=0, batch=8, rows=8, list=0x50000, scale=0.1, sinks=0, scales=(1.0, 1.0), out=0x60000,
             os=(4096, 128), lse=0, scratch=0x100000, bytes=None)
    a.update(over)
    return lib.pa_sparse_attend(ctypes.byref(p) if p is not None else None, ptr(a["q"]), *a["qs"], ptr(a["k"]),
                                ptr(a["v"]), *a["kvs"], a["pages"], ptr(a["bt"]), a["bts"], ptr(a["lens"]),
                                ptr(a["qsl"]), a["batch"], a["rows"], ptr(a["list"]), a["scale"], ptr(a["sinks"]),
                                *a["scales"], None, None, ptr(a["out"]), *a["os"], ptr(a["lse"]), ptr(a["scratch"]),
                                (p.scratch_bytes if p is not None else 0) if a["bytes"] is None else a["bytes"], None)


COMMON = [
    (dict(batch=-1, rows=-1), INVALID), (dict(batch=65, rows=65), INVALID), (dict(rows=7), INVALID),
    (dict(rows=65, qsl=0x70000), INVALID), (dict(scratch=0), INVALID), (dict(scratch=0x100080), UNSUPPORTED),
    (dict(bytes=65536), SMALL), (dict(bt=0), INVALID), (dict(lens=0), INVALID), (dict(bts=2047), INVALID),
    (dict(q=0), INVALID), (dict(pages=0), INVALID), (dict(qs=(0, 128)), INVALID), (dict(batch=0, rows=0), OK),
]


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(bounds=0), INVALID), (dict(out=0), INVALID), (dict(bs=(2048, -256)), INVALID), (dict(q=0x10008), UNSUPPORTED),
    (dict(qs=(4096, 132)), UNSUPPORTED), (dict(bounds=0x20008), UNSUPPORTED), (dict(bs=(2052, 256)), UNSUPPORTED)])
def test_select_refusals(lib, over, status):
    assert select_args(lib, plan(), **over) == status


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(list=0), INVALID), (dict(out=0), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(sinks=0x80000), INVALID), (dict(scales=(1.0, float("nan"))), INVALID),
    (dict(kvs=(16384, 1024, -128)), INVALID), (dict(os=(4096, 0)), INVALID), (dict(q=0x10002), UNSUPPORTED),
    (dict(os=(4097, 128)), UNSUPPORTED), (dict(k=0x20008), UNSUPPORTED), (dict(kvs=(16388, 1024, 128)), UNSUPPORTED),
    (dict(lse=0x90002), UNSUPPORTED)])
def test_attend_refusals(lib, over, status):
    assert attend_args(lib, plan(), **over) == status


def test_attend_needs_the_sinks_of_its_plan(lib):
    assert attend_args(lib, plan(has_sinks=True)) == INVALID


def test_no_plan(lib):
    assert select_args(lib, None) == INVALID and attend_args(lib, None) == INVALID


@pytest.mark.parametrize("edit", [
    lambda p: setattr(p, "scratch_bytes", 65536), lambda p: setattr(p, "score_rows", 1 << 20),
    lambda p: setattr(p, "score_rows", 0), lambda p: setattr(p, "partial_rows", -1),
    lambda p: setattr(p.shape, "max_pages_per_seq", 60000), lambda p: setattr(p.shape, "head_dim", 100),
    lambda p: setattr(p.shape, "num_sms", 0), lambda p: setattr(p.shape, "last_pages", 0)])
def test_hand_edited_plans_are_refused(lib, edit):
    p = plan()
    edit(p)
    assert select_args(lib, p, bytes=1 << 40, bts=60000) == INVALID
    assert attend_args(lib, p, bytes=1 << 40, bts=60000) == INVALID


def test_edited_splits_and_tiles_are_refused(lib):
    p = plan(num_splits=2)
    p.shape.num_splits = 7                       # partials beyond partial_rows
    assert attend_args(lib, p, batch=64, rows=64) == INVALID
    p = plan()
    p.tile_tokens = 64
    assert attend_args(lib, p) == INVALID


def test_binding_refuses_tensors_of_another_kind(lib):
    p = plan()
    cpu = torch.zeros(8, 32, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        pb.select_pages(p, cpu, None, None, None, None, scratch=None)
    with pytest.raises(ValueError, match="rot_dim"):
        pb.rope(rot_dim=64)
    with pytest.raises(ValueError, match="axes"):
        pb.rope(rot_dim=0, sections=(0,) * 5)


def test_device_code_and_exports_match_the_header(lib):
    src = open(os.path.join(ROOT, "include", "pa.h")).read()
    assert int(re.search(r"PA_DEVICE_POSITION\s*=\s*(\d+)", src).group(1)) == pb.DEVICE_POSITION
    for n in ("pa_append_rope_kv", "pa_page_bounds", "pa_sparse_plan", "pa_select_pages", "pa_sparse_attend"):
        assert n in pb.EXPORTED_SYMBOLS and hasattr(lib, n)


def test_structs_have_the_sizes_c_gives_them(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "pa.h"\nint main(void) { printf("%zu %zu %zu\\n", sizeof(pa_rope), '
                   'sizeof(pa_sparse_shape), sizeof(pa_sparse_plan_t)); return 0; }\n')
    exe = tmp_path / "sizes"
    subprocess.run([cc, "-std=c11", "-Wall", "-Wextra", "-Werror", "-I" + os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(pb.PaRope), ctypes.sizeof(pb.PaSparseShape), ctypes.sizeof(pb.PaSparsePlan)]


def test_binding_refuses_workspaces_of_another_kind():
    with pytest.raises(ValueError, match="scratch"):
        pb._scratch(torch.zeros(1 << 17, dtype=torch.uint8), 0)
    with pytest.raises(ValueError, match="scratch"):
        pb._header(torch.zeros(1 << 17, dtype=torch.uint8), 0)
    with pytest.raises(ValueError, match="header"):
        pb._header(torch.zeros(64, dtype=torch.uint8), -1)
    assert pb._header(None, 0) is None


def test_splits_just_above_one_wave_of_ctas(lib):
    # 100 rows of 8 kv heads on 760 (608: e4m3, heads of 128, 80 rows) CTAs: three splits fill the second wave; the
    # 64-key stages of e4m3 heads of 64 are not cut so finely and stay whole
    def partials(rows, **over):
        return plan(max_total_q=rows, max_batch=rows, **over).partial_rows
    assert partials(100) == 300 and partials(80, kv_dtype=1) == 240 and partials(100, head_dim=64) == 300
    assert partials(100, head_dim=64, kv_dtype=1) < 100
    assert partials(95) < 100                        # no more than one wave
