"""pa_append_blocks against the definition: codes and scales must be equal, every code."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from paged_kv_gqa_12_gb300 import binding as pb  # noqa: E402
from tests import block_refs as ref  # noqa: E402

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def _codes(shape, kind, g):
    if kind == "int8":
        return torch.randint(-127, 128, shape, generator=g).to(torch.int8)
    x = (torch.randn(shape, generator=g) * 120).clamp(-448, 448)
    return x.to(ref.E4M3).view(torch.uint8)


def _problem(seed, kind, Hkv, D, ps, ctx, new, spread=2.0, strided=False):
    g = torch.Generator().manual_seed(seed)
    seq = [c + n for c, n in zip(ctx, new)]
    pages = [-(-L // ps) for L in seq]
    pool = sum(pages) + 4
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    table = torch.full((len(ctx), max(pages + [1]) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    qsl = [0]
    for n in new:
        qsl.append(qsl[-1] + n)
    T = qsl[-1]
    kv = torch.randn(T, 2 * Hkv, D, generator=g) * torch.exp(torch.randn(T, 2 * Hkv, 1, generator=g) * 0.5)
    s = dict(kind=kind, ps=ps, seq=seq, qsl=qsl, table=table, kv=kv.bfloat16(), Hkv=Hkv,
             k_scales=0.03 * spread ** (2 * torch.rand(pool, Hkv, generator=g) - 1),
             v_scales=0.03 * spread ** (2 * torch.rand(pool, Hkv, generator=g) - 1))
    s["k_cache"], s["v_cache"] = _codes((pool, ps, Hkv, D), kind, g), _codes((pool, ps, Hkv, D), kind, g)
    return s


def _run(s, decode=False, scratch=None):
    H = s["Hkv"]
    kv = s["kv"].cuda()
    d = {k: s[k].cuda() for k in ("k_cache", "v_cache", "k_scales", "v_scales", "table")}
    seq = torch.tensor(s["seq"], dtype=torch.int32, device="cuda")
    qsl = torch.tensor(s["qsl"], dtype=torch.int32, device="cuda")
    scratch = torch.zeros(pb.SCRATCH_HEADER_BYTES, dtype=torch.uint8, device="cuda") if scratch is None else scratch
    pb.append_blocks(kv[:, :H], kv[:, H:], d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"], d["table"], seq,
                     query_start_loc=None if decode else qsl, scratch=scratch)
    return {k: v.cpu() for k, v in d.items()}, pb.check(scratch)


def _same(s, got):
    H = s["Hkv"]
    for name, x in (("k", s["kv"][:, :H]), ("v", s["kv"][:, H:])):
        v, sc = ref.append(s["kind"], x, s[name + "_cache"], s[name + "_scales"], s["table"], s["seq"], s["qsl"], s["ps"])
        a = ref.values(got[name + "_cache"])
        assert torch.equal(got[name + "_scales"], sc), name
        assert torch.equal(a.nan_to_num(nan=1e9), v.nan_to_num(nan=1e9)), (name, (a != v).sum())


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ps", [16, 32, 64])
def test_every_form(kind, D, ps):
    ctx = [0, 0, 1, ps - 1, ps, ps + 1, 5, 0, 3 * ps - 2, 40]
    new = [1, ps, 1, 1, 3, ps - 1, 0, 0, 2 * ps + 5, 3]
    s = _problem(D + ps, kind, 2, D, ps, ctx, new)
    got, code = _run(s)
    assert code == 0
    _same(s, got)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("B,Hkv", [(1, 1), (2, 8), (70, 3), (300, 8)])
def test_decode(kind, B, Hkv):
    s = _problem(B, kind, Hkv, 128, 16, [(i * 37) % 100 for i in range(B)], [1] * B)
    got, code = _run(s, decode=True)
    assert code == 0
    _same(s, got)


def test_decode_of_a_padded_batch():
    # requests of length 0 bring nothing, and are no error
    s = _problem(31, "int8", 2, 128, 16, [30, 0, 5, 0], [1, 1, 1, 1])
    s["seq"][1] = s["seq"][3] = 0
    got, code = _run(s, decode=True)
    assert code == 0
    H = s["Hkv"]
    for name, x in (("k", s["kv"][:, :H]), ("v", s["kv"][:, H:])):
        v, sc = ref.append("int8", x[[0, 2]], s[name + "_cache"], s[name + "_scales"], s["table"][[0, 2]], [31, 6],
                           [0, 1, 2], 16)
        assert torch.equal(ref.values(got[name + "_cache"]), v) and torch.equal(got[name + "_scales"], sc)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_many_rows(kind):
    s = _problem(3, kind, 8, 128, 16, [0, 300, 17, 0, 1000, 3], [700, 1, 1200, 0, 333, 16])
    got, code = _run(s)
    assert code == 0
    _same(s, got)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_ties_round_to_even(kind):
    # scale 1 exactly: halves are ties; and a scale of 3 / 127 whose quotients are next to ties
    most = ref.MOST[kind]
    s = _problem(4, kind, 1, 64, 16, [0, 0], [16, 16])
    x = torch.arange(16 * 128).reshape(16, 2, 64) * 0.5 - 256
    x = x.clamp(-most, most)
    x[0, :, 0] = most
    y = (torch.arange(16 * 128).reshape(16, 2, 64) % 301 - 150) / 64.0
    y[0, :, 0] = 3.0
    s["kv"] = torch.cat([x, y.clamp(-3, 3)]).bfloat16()
    got, _ = _run(s)
    _same(s, got)
    assert float(got["k_scales"][s["table"][0, 0], 0]) == 1.0


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_all_quotients_of_a_scale(kind):
    # every positive bf16 number below the largest, by scales of all mantissas' neighbourhoods: rounding is exact
    s = _problem(5, kind, 2, 256, 64, [0] * 40, [64] * 40)
    g = torch.Generator().manual_seed(9)
    bits = torch.randint(0x3c00, 0x4180, (64 * 40, 4, 256), generator=g).to(torch.int16)
    s["kv"] = bits.view(torch.bfloat16)
    got, _ = _run(s)
    _same(s, got)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_zeros_infinities_nan_and_tiny_values(kind):
    s = _problem(6, kind, 2, 64, 16, [0, 0, 3, 20, 0], [16, 5, 2, 4, 3])
    kv = s["kv"]
    kv[:16] = 0                                            # a page of zeros: scale 0
    kv[17, 0, 3], kv[18, 1, 4], kv[19, 2, 5] = float("inf"), float("-inf"), float("nan")
    kv[21, 0] = float("nan")                               # (all of one head's new row)
    kv[23:27] *= 2.0 ** -126                               # next to the smallest numbers
    kv[27:30] *= 2.0 ** 120
    got, code = _run(s)
    assert code == 0
    _same(s, got)
    assert float(got["k_scales"][s["table"][0, 0]].max()) == 0.0


def test_growing_scale_keeps_what_is_beyond_the_page_and_request():
    s = _problem(7, "int8", 4, 128, 16, [10, 26], [1, 1], spread=1.0)
    s["kv"] *= 8                                           # far beyond the old scales: older codes are rounded again
    got, _ = _run(s)
    _same(s, got)
    page = int(s["table"][0, 0])
    assert torch.equal(got["k_cache"][page, 11:], s["k_cache"][page, 11:])     # slots behind the new token stay


def test_requests_that_do_not_fit_stay_unwritten():
    s = _problem(8, "int8", 2, 64, 16, [3, 8, 2, 5], [4, 4, 4, 4])
    s["seq"][1] = 3                                        # more new tokens than the length
    s["seq"][2] = s["table"].shape[1] * 16 + 1             # beyond the table
    want = dict(s, seq=[s["seq"][0], 0, 0, s["seq"][3]])
    got, code = _run(s)
    assert code == pb.DEVICE_CAPACITY
    H = s["Hkv"]
    for name, x in (("k", s["kv"][:, :H]), ("v", s["kv"][:, H:])):
        # (the reference passes over requests 1 and 2: their packed rows are skipped by emptying them)
        a, sc = s[name + "_cache"].clone(), s[name + "_scales"].clone()
        v = ref.values(a)
        for b in (0, 3):
            one = dict(table=s["table"][b:b + 1], seq=[s["seq"][b]], qsl=[0, 4])
            v2, sc = ref.append("int8", x[4 * b:4 * b + 4], a, sc, one["table"], one["seq"], one["qsl"], 16)
            a = v2.to(torch.int8)
            v = v2
        assert torch.equal(ref.values(got[name + "_cache"]), v) and torch.equal(got[name + "_scales"], sc)
    assert want["seq"][1] == 0


def test_pages_outside_the_pool_are_passed_over():
    s = _problem(9, "e4m3", 2, 64, 16, [0, 20], [40, 3])
    s["table"][0, 1] = s["k_cache"].shape[0]
    s["table"][1, 1] = -1
    got, code = _run(s)
    assert code == pb.DEVICE_PAGE_ID
    mid = {int(s["table"][0, 0]), int(s["table"][0, 2])}
    for p in range(s["k_cache"].shape[0]):
        if p not in mid:
            assert torch.equal(got["k_cache"][p], s["k_cache"][p]) and torch.equal(got["v_scales"][p], s["v_scales"][p])


def test_strides_and_rows_behind_the_last():
    # caches that are halves of one allocation, heads first, scales with padded rows; rows behind the last request
    s = _problem(10, "int8", 4, 128, 32, [5, 64, 0], [3, 40, 1])
    T, H, D, ps = s["qsl"][-1], 4, 128, 32
    pool = s["k_cache"].shape[0]
    both = torch.zeros(pool, 2, H, ps, D, dtype=torch.int8, device="cuda")
    k, v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    k.copy_(s["k_cache"]); v.copy_(s["v_cache"])
    sc = torch.full((pool, 2 * H + 3), 9.0, device="cuda")
    ks, vs = sc[:, :H], sc[:, H:2 * H]
    ks.copy_(s["k_scales"]); vs.copy_(s["v_scales"])
    new = torch.full((T + 5, 2 * H + 1, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    new[:T, :2 * H] = s["kv"].cuda()
    pb.append_blocks(new[:, :H], new[:, H:2 * H], k, v, ks, vs, s["table"].cuda(),
                     torch.tensor(s["seq"], dtype=torch.int32, device="cuda"),
                     query_start_loc=torch.tensor(s["qsl"], dtype=torch.int32, device="cuda"))
    _same(s, dict(k_cache=k.contiguous().cpu(), v_cache=v.contiguous().cpu(), k_scales=ks.cpu(), v_scales=vs.cpu()))
    assert torch.equal(sc[:, 2 * H:], torch.full_like(sc[:, 2 * H:], 9.0))


def test_a_pool_beyond_32_bits():
    # page offsets above 2^32 bytes
    H, D, ps = 8, 256, 64
    pool = (1 << 32) // (H * D * ps) + 40
    k = torch.empty(pool, ps, H, D, dtype=torch.int8, device="cuda")
    v = torch.empty_like(k)
    ks, vs = torch.ones(pool, H, device="cuda"), torch.ones(pool, H, device="cuda")
    table = torch.tensor([[pool - 1, 0], [3, pool - 20]], dtype=torch.int32)
    s = _problem(12, "int8", H, D, ps, [0, 0], [70, 100])
    kv = s["kv"].cuda()
    for t in (k, v):
        for i in (pool - 1, 0, 3, pool - 20):
            t[i] = 0
    pb.append_blocks(kv[:, :H], kv[:, H:], k, v, ks, vs, table.cuda(),
                     torch.tensor([70, 100], dtype=torch.int32, device="cuda"),
                     query_start_loc=torch.tensor([0, 70, 170], dtype=torch.int32, device="cuda"))
    ids = [pool - 1, 0, 3, pool - 20]
    small = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    for t, sc, x in ((k, ks, s["kv"][:, :H]), (v, vs, s["kv"][:, H:])):
        want, wsc = ref.append("int8", x, torch.zeros(4, ps, H, D, dtype=torch.int8), torch.ones(4, H), small, [70, 100],
                               [0, 70, 170], ps)
        got = torch.stack([t[i] for i in ids]).cpu()
        assert torch.equal(ref.values(got), want) and torch.equal(sc[ids].cpu(), wsc)
