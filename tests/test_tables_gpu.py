"""pa_step_tables against an allocator that hands out pages one by one: every output is a whole
number and must be equal."""
import random

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from paged_kv_gqa_12_gb300 import binding as pb  # noqa: E402
from tests import block_refs as ref  # noqa: E402

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def _state(seed, B, ps, ctx_hi, new_hi, ended=0.2, spare=9, pad=5):
    """Requests with random contexts, held pages (some more than they need) and new tokens; a shuffled pool."""
    rng = random.Random(seed)
    ctx = [rng.randint(0, ctx_hi) for _ in range(B)]
    new = [-1 if rng.random() < ended else rng.choice([0, 1, 1, rng.randint(0, new_hi)]) for _ in range(B)]
    held = [-(-c // ps) + rng.choice([0, 0, 1, 3]) for c in ctx]
    width = max([h for h in held] + [-(-(c + max(n, 0)) // ps) for c, n in zip(ctx, new)] + [1]) + 1
    back = sum(h for h, n in zip(held, new) if n < 0)
    need = sum(max(0, -(-(c + n) // ps) - h) for c, n, h in zip(ctx, new, held) if n >= 0)
    pool = sum(held) + max(0, need - back) + spare
    perm = list(range(pool))
    rng.shuffle(perm)
    table = torch.full((B, width), -7, dtype=torch.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = torch.tensor(perm[at:at + h], dtype=torch.int32)
        at += h
    free = torch.full((pool,), -9, dtype=torch.int32)
    free[:pool - at] = torch.tensor(perm[at:], dtype=torch.int32)
    return dict(ctx=ctx, new=new, held=held, table=table, free=free, count=pool - at, pool=pool, ps=ps,
                tokens=sum(max(n, 0) for n in new) + pad)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _upload(s):
    B = len(s["ctx"])
    d = dict(ctx=_i32(s["ctx"]), new=_i32(s["new"]), held=_i32(s["held"]), table=s["table"].cuda(),
             free=s["free"].cuda(), count=_i32([s["count"]]))
    d["seq"], d["qsl"] = torch.full((B,), 77, **_k), torch.full((B + 1,), 77, **_k)
    d["slots"] = torch.full((s["tokens"],), 77, dtype=torch.int64, device="cuda")
    d["pos"] = torch.full((s["tokens"],), 77, **_k)
    d["scratch"] = torch.zeros(pb.SCRATCH_HEADER_BYTES, dtype=torch.uint8, device="cuda")
    return d


_k = dict(dtype=torch.int32, device="cuda")


def _call(s, d, **kw):
    pb.step_tables(d["ctx"], d["new"], d["held"], d["free"], d["count"], d["table"], page_size=s["ps"],
                   num_pages=s["pool"], seq_lens=d["seq"], query_start_loc=d["qsl"], slots=d["slots"],
                   positions=d["pos"], **{**dict(scratch=d["scratch"]), **kw})


def _check(s, d, held, count):
    want = ref.tables(s["ctx"], s["new"], s["held"], s["free"], s["count"], s["table"], s["ps"], s["tokens"])
    table, free, n, counts, seq, qsl, slots, pos = want
    assert torch.equal(d["table"].cpu(), table)
    assert torch.equal(d["free"].cpu()[:n], free[:n])
    # entries above the stack are leftovers; those below the old count that were not handed out stay
    assert int(count) == n and held.tolist() == counts
    assert d["seq"].tolist() == seq and d["qsl"].tolist() == qsl
    assert d["slots"].tolist() == slots and d["pos"].tolist() == pos


@pytest.mark.parametrize("B,ps,ctx_hi,new_hi,ended", [
    (1, 16, 0, 1, 0.0), (1, 16, 40, 1, 1.0), (3, 16, 15, 40, 0.0), (7, 64, 300, 5, 0.3), (33, 32, 200, 90, 0.5),
    (250, 16, 1000, 30, 0.1), (513, 16, 60, 40, 0.2), (1500, 1, 9, 3, 0.3), (8192, 16, 30, 4, 0.2), (40, 24, 500, 700, 0.2)])
@pytest.mark.parametrize("inplace", [False, True])
def test_matches_the_allocator(B, ps, ctx_hi, new_hi, ended, inplace):
    for seed in range(3):
        s = _state(1000 * B + seed, B, ps, ctx_hi, new_hi, ended)
        d = _upload(s)
        if inplace:
            _call(s, d)
            held, count = d["held"], d["count"]
        else:
            held, count = torch.full((B,), 5, **_k), torch.full((1,), 5, **_k)
            _call(s, d, page_counts_out=held, free_count_out=count)
            assert d["held"].tolist() == s["held"] and int(d["count"]) == s["count"]
        assert pb.check(d["scratch"]) == 0
        _check(s, d, held, count)


def test_lengths_in_place():
    # seq_lens over context_lens, as a server that keeps one array of lengths calls it
    s = _state(5, 300, 16, 400, 60)
    d = _upload(s)
    d["seq"] = d["ctx"]
    _call(s, d)
    _check(s, d, d["held"], d["count"])


def test_steps_in_a_row_return_every_page():
    # requests come, grow and end: the pool's pages stay a permutation, and all come back
    rng = random.Random(11)
    B, ps, pool, W = 40, 16, 400, 40
    ctx, held = [0] * B, [0] * B
    d = dict(ctx=_i32(ctx), held=_i32(held), table=torch.full((B, W), -1, **_k), free=_i32(list(range(pool))),
             count=_i32([pool]), scratch=torch.zeros(pb.SCRATCH_HEADER_BYTES, dtype=torch.uint8, device="cuda"))
    seq, qsl = torch.empty(B, **_k), torch.empty(B + 1, **_k)
    slots, pos = torch.empty(2000, dtype=torch.int64, device="cuda"), torch.empty(2000, **_k)
    for step in range(30):
        new = [-1 if (rng.random() < 0.2 or c > 120 or step == 29) else rng.choice([0, 1, 1, 4, 30]) for c in ctx]
        d["new"] = _i32(new)
        pb.step_tables(d["ctx"], d["new"], d["held"], d["free"], d["count"], d["table"], page_size=ps, num_pages=pool,
                       seq_lens=seq, query_start_loc=qsl, slots=slots, positions=pos, scratch=d["scratch"])
        ctx = [0 if n < 0 else c + n for c, n in zip(ctx, new)]
        assert seq.tolist() == ctx
        d["ctx"].copy_(seq)
        held, count, table = d["held"].tolist(), int(d["count"]), d["table"].cpu()
        owned = [int(table[b, i]) for b in range(B) for i in range(held[b])] + d["free"].tolist()[:count]
        assert sorted(owned) == list(range(pool))
        assert all(h * ps >= c for h, c in zip(held, ctx))
        got = [x for x in slots.tolist() if x >= 0]
        assert len(set(got)) == len(got) == sum(max(n, 0) for n in new)
    assert pb.check(d["scratch"]) == 0 and int(d["count"]) == pool


@pytest.mark.parametrize("what", ["pages", "tokens", "width", "negative", "context", "count", "held", "below"])
def test_a_step_that_does_not_fit_changes_nothing(what):
    s = _state(21, 60, 16, 300, 50, ended=0.0 if what == "pages" else 0.2)
    bit = pb.DEVICE_CAPACITY
    if what == "pages":
        s["new"] = [60] * 60
        s["tokens"] = 4000
        s["table"] = torch.nn.functional.pad(s["table"], (0, 5), value=-7)
        bit = pb.DEVICE_NO_PAGES
    elif what == "tokens":
        s["tokens"] = sum(max(n, 0) for n in s["new"]) - 1
    elif what == "width":
        s["ctx"][30] = s["table"].shape[1] * 16
        s["held"][30] = s["table"].shape[1]
        s["new"][30] = 1
    elif what == "negative":
        s["new"][59] = -2
    elif what == "context":
        s["ctx"][7], s["held"][7], s["new"][7] = 33, 2, 1
    elif what == "count":
        s["count"] = s["pool"] + 1
    elif what == "held":
        s["held"][0] = s["table"].shape[1] + 1
    else:
        s["ctx"][3] = -1
    d = _upload(s)
    held, count = torch.full((60,), 5, **_k), torch.full((1,), 5, **_k)
    _call(s, d, page_counts_out=held, free_count_out=count)
    assert pb.check(d["scratch"]) == bit
    assert torch.equal(d["table"].cpu(), s["table"]) and torch.equal(d["free"].cpu(), s["free"])
    assert held.tolist() == s["held"] and int(count) == s["count"]
    assert d["seq"].tolist() == s["ctx"] and d["qsl"].tolist() == [0] * 61
    assert set(d["slots"].tolist()) == {-1} and set(d["pos"].tolist()) == {0}


def test_bad_page_ids_become_padding():
    s = _state(31, 20, 16, 100, 20, ended=0.0)
    s["ctx"][4], s["held"][4], s["new"][4] = 5, max(1, s["held"][4]), 3
    s["table"][4, 0] = s["pool"]
    d = _upload(s)
    _call(s, d)
    assert pb.check(d["scratch"]) == pb.DEVICE_PAGE_ID
    at = d["qsl"].tolist()[4]
    assert d["slots"].tolist()[at:at + 3] == [-1, -1, -1] and d["pos"].tolist()[at:at + 3] == [5, 6, 7]
    assert min(d["slots"].tolist()[:at]) >= 0 if at else True


def test_no_requests_and_no_tokens():
    d = dict(z=torch.zeros(0, **_k))
    qsl, count, slots, pos = torch.full((1,), 9, **_k), _i32([3]), torch.full((4,), 7, dtype=torch.int64,
                                                                                device="cuda"), torch.full((4,), 7, **_k)
    pb.step_tables(d["z"], d["z"], d["z"], _i32([0, 1, 2]), count, torch.zeros(0, 1, **_k), page_size=16, num_pages=3,
                   seq_lens=d["z"], query_start_loc=qsl, slots=slots, positions=pos)
    assert qsl.tolist() == [0] and int(count) == 3 and slots.tolist() == [-1] * 4


def test_replayed_graph():
    s = _state(41, 250, 16, 1000, 30)
    d = _upload(s)
    held, count = torch.zeros(250, **_k), torch.zeros(1, **_k)
    _call(s, d, page_counts_out=held, free_count_out=count)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _call(s, d, page_counts_out=held, free_count_out=count)
    t = _state(42, 250, 16, 700, 20)
    if t["table"].shape[1] > s["table"].shape[1] or t["pool"] > s["pool"] or t["tokens"] > s["tokens"]:
        pytest.fail("the second batch must fit the first one's buffers")
    d["ctx"].copy_(_i32(t["ctx"])); d["new"].copy_(_i32(t["new"])); d["held"].copy_(_i32(t["held"]))
    d["table"][:, :t["table"].shape[1]] = t["table"].cuda()
    d["free"][:t["pool"]] = t["free"].cuda()
    d["count"].copy_(_i32([t["count"]]))
    t["tokens"], t["table"], t["pool"] = s["tokens"], d["table"].cpu(), s["pool"]
    t["free"] = d["free"].cpu()
    g.replay()
    torch.cuda.synchronize()
    _check(t, d, held, count)
