"""pa_append_rope_kv against its definition in 64 bits: norms, rotations of one
and several axes, both cache types, strides, padding, bad slots and positions."""
import pytest
import torch

from tests import long_refs as lr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_12_gb300 import binding
    binding.load()
    return binding


def table(max_pos, rot):
    f = 1e4 ** (-torch.arange(0, max(rot, 1), 2, dtype=torch.float64) / max(rot, 1))[:rot // 2]
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def make(T, Hq, Hkv, D, ps, *, kv, axes=1, sections=None, rot=None, norm=True, seed=0, max_pos=4096,
         interleaved=False, layout="separate"):
    g = torch.Generator().manual_seed(seed)
    rot = D if rot is None else rot
    d = dict(T=T, Hq=Hq, Hkv=Hkv, D=D, ps=ps, kv=kv, rot=rot, interleaved=interleaved)
    d["sections"] = sections or (rot // 2,)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).bfloat16()
    d["q"], d["k"], d["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pool = -(-T // ps) + 3
    dt = torch.uint8 if kv == "e4m3" else torch.bfloat16
    if layout == "separate":
        d["kc"] = torch.randint(0, 120, (pool, ps, Hkv, D), generator=g).to(dt)
        d["vc"] = torch.randint(0, 120, (pool, ps, Hkv, D), generator=g).to(dt)
    else:
        both = torch.randint(0, 120, (pool, 2, ps, Hkv, D), generator=g).to(dt)
        d["kc"], d["vc"] = both[:, 0], both[:, 1]
    d["slots"] = torch.randperm(pool * ps, generator=g)[:T]
    d["pos"] = torch.randint(0, max_pos, (axes, T), generator=g).to(torch.int32)
    d["table"] = table(max_pos, rot)
    d["wq"] = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16() if norm else None
    d["wk"] = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16() if norm else None
    d["scale"] = (0.02, 0.03) if kv == "e4m3" else (1.0, 1.0)
    d["eps"], d["offset"] = 1e-5, 0.0
    return d


def cuda(t):
    """On the GPU with the same strides (views of one storage stay views of their shape)."""
    if t is None:
        return None
    base = torch.empty(t.untyped_storage().nbytes() // t.element_size(), dtype=t.dtype)
    base = torch.as_strided(t, (base.numel(),), (1,), 0).cuda()
    return torch.as_strided(base, t.shape, t.stride(), t.storage_offset())


def run(pb, d, *, scratch=None, q=True, inplace=False, stream=None):
    r = pb.rope(None if d["rot"] == 0 else cuda(d["table"]), rot_dim=d["rot"], interleaved=d["interleaved"],
                sections=None if len(d["sections"]) == 1 else d["sections"], q_norm=cuda(d["wq"]), k_norm=cuda(d["wk"]),
                norm_eps=d["eps"], norm_offset=d["offset"])
    kc, vc = cuda(d["kc"]), cuda(d["vc"])
    qi = cuda(d["q"]) if q else None
    qo = qi if inplace else torch.full(d["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda") if q else None
    pb.append_rope_kv(r, cuda(d["k"]), cuda(d["v"]), cuda(d["pos"]) if d["rot"] else None, kc, vc, cuda(d["slots"]),
                      q=qi, q_out=qo, kv_dtype=pb.KV_FP8_E4M3 if d["kv"] == "e4m3" else pb.KV_BF16,
                      k_scale=d["scale"][0], v_scale=d["scale"][1], scratch=scratch, stream=stream)
    torch.cuda.synchronize()
    return (qo.cpu() if q else None), kc.cpu(), vc.cpu()


def expect(d):
    kw = dict(positions=d["pos"], table=d["table"], rot=d["rot"], interleaved=d["interleaved"], sections=d["sections"],
              eps=d["eps"], offset=d["offset"])
    return lr.norm_rotate(d["q"], d["wq"], **kw), lr.norm_rotate(d["k"], d["wk"], **kw)


def near(got, want, size, half, least=0.0):
    """Within half a step of the result's type, and 2^-18 of the pair for the 32-bit norm and rotation (a sum of up
    to 256 squares in 12 steps, a reciprocal root of 2 units, three products and a sum: below 2^-19)."""
    err = (got.double() - want).abs()
    tol = half * want.abs() + 2.0 ** -18 * size + least
    assert (err <= tol).all(), f"off by {(err - tol).max():.3e}"


def check(d, got, rows=None):
    q, kc, vc = got
    (yq, mq), (yk, mk) = expect(d)
    rows = torch.arange(d["T"]) if rows is None else rows
    if q is not None:
        near(q[rows], yq[rows], mq[rows], 2.0 ** -8)
    page, slot = d["slots"][rows] // d["ps"], d["slots"][rows] % d["ps"]
    if d["kv"] == "bf16":
        near(kc[page, slot], yk[rows], mk[rows], 2.0 ** -8)
        assert torch.equal(vc[page, slot].view(torch.int16), d["v"][rows].contiguous().view(torch.int16))
    else:
        want = (yk[rows] / d["scale"][0]).clamp(-448, 448)
        # subnormal steps of e4m3 are 2^-9 wide
        near(kc[page, slot].view(torch.float8_e4m3fn), want, mk[rows] / d["scale"][0], 2.0 ** -4, 2.0 ** -10)
        v = (d["v"][rows].float() / torch.tensor(d["scale"][1])).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(vc[page, slot], v.view(torch.uint8))
    # every other slot is as it was
    for new, old in ((kc, d["kc"]), (vc, d["vc"])):
        rest = torch.ones(old.shape[:2], dtype=torch.bool)
        rest[page, slot] = False
        assert torch.equal(new[rest], old[rest])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,ps", [(8, 2, 64, 16), (32, 8, 128, 16), (16, 8, 256, 32), (7, 1, 64, 64), (5, 5, 128, 16)])
@pytest.mark.parametrize("norm", [False, True])
def test_matches_definition(pb, kv, Hq, Hkv, D, ps, norm):
    for T in (1, 3, 77):
        d = make(T, Hq, Hkv, D, ps, kv=kv, norm=norm, seed=T + D)
        check(d, run(pb, d))


@pytest.mark.parametrize("D,rot,interleaved", [(128, 64, False), (128, 64, True), (64, 64, True), (256, 8, False),
                                               (256, 104, True), (64, 40, False), (128, 0, False)])
def test_partial_and_interleaved(pb, D, rot, interleaved):
    for kv in ("bf16", "e4m3"):
        d = make(33, 6, 2, D, 16, kv=kv, rot=rot, interleaved=interleaved, seed=rot)
        check(d, run(pb, d))


@pytest.mark.parametrize("sections", [(16, 24, 24), (1, 2, 61), (0, 64), (5, 9, 3, 47), (64, 0, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_axes(pb, sections, interleaved):
    d = make(50, 8, 2, 128, 16, kv="bf16", axes=len(sections), sections=sections, interleaved=interleaved, seed=sum(sections[:2]))
    check(d, run(pb, d))


def test_norm_of_one_side_and_offset(pb):
    for drop in ("wq", "wk"):
        d = make(20, 4, 4, 128, 16, kv="bf16", seed=5)
        d[drop] = None
        d["offset"], d["eps"] = 1.0, 0.0
        check(d, run(pb, d))


def test_far_positions(pb):
    d = make(64, 8, 2, 128, 16, kv="bf16", max_pos=200000, seed=6)
    d["pos"][0, :5] = torch.tensor([199999, 0, 131071, 131072, 65536])
    check(d, run(pb, d))


def test_keys_alone_and_in_place(pb):
    d = make(40, 8, 2, 64, 16, kv="e4m3", seed=7)
    check(d, run(pb, d, q=False))
    check(d, run(pb, d, inplace=True))


def test_interleaved_cache_layout(pb):
    for kv in ("bf16", "e4m3"):
        d = make(90, 8, 4, 128, 32, kv=kv, layout="interleaved", seed=8)
        check(d, run(pb, d))


def test_padding_and_bad_tokens_are_untouched(pb):
    d = make(60, 8, 2, 128, 16, kv="bf16", seed=9)
    pool = d["kc"].shape[0]
    skip = torch.zeros(60, dtype=torch.bool)
    d["slots"][::7] = -1
    skip[::7] = True
    scratch = torch.zeros(pb.SCRATCH_HEADER_BYTES, dtype=torch.uint8, device="cuda")
    got = run(pb, d, scratch=scratch)
    assert pb.check(scratch) == 0
    assert (got[0][skip] == 7.0).all()
    check(d, got, torch.arange(60)[~skip])
    d["slots"][1] = pool * d["ps"]            # just behind the pool
    skip[1] = True
    got = run(pb, d, scratch=scratch)
    assert pb.check(scratch) == pb.DEVICE_PAGE_ID
    assert (got[0][skip] == 7.0).all()
    check(d, got, torch.arange(60)[~skip])
    d["slots"][1] = -1
    d["pos"][0, 2], d["pos"][0, 3] = -1, 4096
    skip[2] = skip[3] = True
    got = run(pb, d, scratch=scratch)
    assert pb.check(scratch) == pb.DEVICE_POSITION
    assert (got[0][skip] == 7.0).all()
    check(d, got, torch.arange(60)[~skip])


def test_infinities_and_nan_stay_in_their_rows(pb):
    d = make(12, 4, 2, 64, 16, kv="bf16", seed=10)
    clean = run(pb, d)
    d["q"][3, 1, 5] = float("nan")
    d["k"][4, 0, 9] = float("inf")
    got = run(pb, d)
    keep = torch.ones(12, 4, dtype=torch.bool)
    keep[3, 1] = False
    assert torch.equal(got[0][keep], clean[0][keep]) and got[0][3, 1].isnan().all()
    page, slot = d["slots"] // 16, d["slots"] % 16
    keep = torch.ones(12, 2, dtype=torch.bool)
    keep[4, 0] = False
    assert torch.equal(got[1][page, slot][keep], clean[1][page, slot][keep])


def test_norm_of_zero_row_is_finite(pb):
    d = make(4, 4, 2, 64, 16, kv="bf16", seed=11)
    d["q"][:] = 0
    d["k"][:] = 0
    check(d, run(pb, d))


def test_pool_beyond_32_bit_offsets(pb):
    # 2.1 billion elements (4.3 GB) a cache: slots whose byte and element offsets pass 32 bits
    Hkv, D, ps = 8, 128, 16
    pages = (1 << 31) // (ps * Hkv * D) + 64
    kc = torch.zeros(pages, ps, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    d = make(5, 8, Hkv, D, ps, kv="bf16", seed=12)
    slots = torch.tensor([0, pages * ps - 1, pages * ps - 17, (pages // 2) * ps, (pages - 40) * ps + 3])
    r = pb.rope(cuda(d["table"]), rot_dim=D, q_norm=cuda(d["wq"]), k_norm=cuda(d["wk"]), norm_eps=d["eps"])
    qo = torch.empty(5, 8, D, dtype=torch.bfloat16, device="cuda")
    pb.append_rope_kv(r, cuda(d["k"]), cuda(d["v"]), cuda(d["pos"]), kc, vc, slots.cuda(), q=cuda(d["q"]), q_out=qo)
    (yq, mq), (yk, mk) = expect(d)
    at = slots.cuda()
    near(kc.view(-1, Hkv, D)[at].cpu(), yk, mk, 2.0 ** -8)
    near(qo.cpu(), yq, mq, 2.0 ** -8)
    assert torch.equal(vc.view(-1, Hkv, D)[at].cpu(), d["v"])
    assert int((kc.view(-1, Hkv * D).abs().amax(1) > 0).sum()) == 5


def test_graph_capture_and_other_stream(pb):
    d = make(30, 8, 2, 128, 16, kv="bf16", seed=13)
    side = torch.cuda.Stream()
    check(d, run(pb, d, stream=side))
    r = pb.rope(cuda(d["table"]), rot_dim=128, q_norm=cuda(d["wq"]), k_norm=cuda(d["wk"]), norm_eps=d["eps"])
    k, v, q, pos, slots = (cuda(d[n]) for n in ("k", "v", "q", "pos", "slots"))
    kc, vc = cuda(d["kc"]), cuda(d["vc"])
    qo = torch.zeros(30, 8, 128, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pb.append_rope_kv(r, k, v, pos, kc, vc, slots, q=q, q_out=qo)
    graph.replay()
    torch.cuda.synchronize()
    check(d, (qo.cpu(), kc.cpu(), vc.cpu()))
    e = make(30, 8, 2, 128, 16, kv="bf16", seed=14)
    for dst, n in ((k, "k"), (v, "v"), (q, "q"), (pos, "pos"), (slots, "slots"), (kc, "kc"), (vc, "vc")):
        dst.copy_(cuda(e[n]))
    graph.replay()
    torch.cuda.synchronize()
    e["wq"], e["wk"], e["table"] = d["wq"], d["wk"], d["table"]
    check(e, (qo.cpu(), kc.cpu(), vc.cpu()))


# Calls of many tokens: a token takes 8, 4, 2 or 1 warps by how many there are (on 152
# SMs 8 up to 608 tokens, 1 beyond 2432), and a CTA several tokens.

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D", [(9, 3, 64), (9, 3, 128), (5, 3, 256)])
@pytest.mark.parametrize("T", [700, 1300, 2500, 5003])
@pytest.mark.parametrize("interleaved,norm", [(False, True), (True, False)])
def test_many_tokens(pb, kv, Hq, Hkv, D, T, interleaved, norm):
    half = D // 2
    d = make(T, Hq, Hkv, D, 16, kv=kv, axes=3, sections=(half // 4, half // 4 + 3, half - half // 2 - 3), norm=norm,
             interleaved=interleaved, seed=T + D, layout="interleaved" if T == 1300 else "separate")
    pad = torch.zeros(T, dtype=torch.bool)
    pad[3::11] = True
    pad[T - 1] = T == 2500
    d["slots"][pad] = -1
    got = run(pb, d)
    assert (got[0][pad] == 7.0).all()
    check(d, got, torch.arange(T)[~pad])


@pytest.mark.parametrize("T", [700, 1300, 2500])
def test_many_tokens_norm_of_one_side_keys_alone_and_in_place(pb, T):
    for drop in ("wq", "wk"):
        d = make(T, 8, 2, 128, 64, kv="bf16", rot=64, seed=T)
        d[drop] = None
        d["offset"] = 1.0
        check(d, run(pb, d, inplace=True))
        check(d, run(pb, d, q=False))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [40, 2600])
@pytest.mark.parametrize("Hq,Hkv,D", [(261, 69, 64), (131, 35, 128), (67, 17, 256)])
def test_heads_that_take_several_rounds(pb, kv, T, Hq, Hkv, D):
    # more heads than a token's warps hold rows of at a time
    if T > 40:
        Hq, Hkv = Hq // 8, Hkv // 8
    d = make(T, Hq, Hkv, D, 16, kv=kv, seed=T + Hq, interleaved=kv == "e4m3")
    check(d, run(pb, d))


def test_many_tokens_with_bad_slots_and_positions(pb):
    T = 2700
    d = make(T, 4, 2, 64, 16, kv="bf16", seed=40)
    skip = torch.zeros(T, dtype=torch.bool)
    for i, (slot, pos) in {5: (-1, 0), 1600: (d["kc"].shape[0] * 16, 0), 2699: (None, 4096), 2000: (None, -1)}.items():
        skip[i] = True
        if slot is None:
            d["pos"][0, i] = pos
        else:
            d["slots"][i] = slot
    scratch = torch.zeros(pb.SCRATCH_HEADER_BYTES, dtype=torch.uint8, device="cuda")
    got = run(pb, d, scratch=scratch)
    assert pb.check(scratch) == pb.DEVICE_PAGE_ID | pb.DEVICE_POSITION
    assert (got[0][skip] == 7.0).all()
    check(d, got, torch.arange(T)[~skip])
