"""pa_verify_tokens against the definition on the host in 64 bits: tokens and counts must be equal."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from paged_kv_gqa_12_gb300 import binding as pb  # noqa: E402
from tests import block_refs as ref  # noqa: E402

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def _problem(seed, rows, V, drafts=True, sharp=2.0, near=0.8):
    g = torch.Generator().manual_seed(seed)
    qsl = [0]
    for n in rows:
        qsl.append(qsl[-1] + n)
    T = qsl[-1]
    logits = sharp * torch.randn(T, V, generator=g)
    p = torch.softmax(logits, -1)
    q = torch.softmax(logits + near * torch.randn(T, V, generator=g), -1)
    drawn = torch.multinomial(q if V > 1 else torch.ones(T, 1), 1, generator=g).flatten().to(torch.int32) if T else torch.zeros(0, dtype=torch.int32)
    tokens = torch.cat([drawn.new_zeros(1), drawn[:-1]]) if T else drawn
    return dict(p=p, q=q if drafts else None, tokens=tokens, qsl=qsl, u=torch.rand(T, generator=g),
                w=torch.rand(len(rows), generator=g), width=max(rows) + 2)


def _run(s, width=None, scratch=None):
    B = len(s["qsl"]) - 1
    out = torch.full((B, width or s["width"]), 99, dtype=torch.int32, device="cuda")
    num = torch.full((B,), 99, dtype=torch.int32, device="cuda")
    c = lambda x: None if x is None else x.cuda()       # noqa: E731
    pb.verify_tokens(c(s["tokens"]), c(s["p"]), torch.tensor(s["qsl"], dtype=torch.int32, device="cuda"), c(s["u"]),
                     c(s["w"]), out, num, draft_probs=c(s["q"]), scratch=scratch)
    return out.cpu(), num.cpu()


def _same(s, got=None):
    out, num = got or _run(s)
    o, n = ref.verify(s["tokens"], s["p"], s["q"], s["qsl"], s["u"], s["w"], s["width"])
    assert torch.equal(num, n), (num, n)
    assert torch.equal(out, o), ((out != o).nonzero()[:5], out[(out != o)][:5], o[(out != o)][:5])


@pytest.mark.parametrize("V", [1, 2, 31, 127, 128, 129, 1000, 4099, 32000, 50001, 131072])
@pytest.mark.parametrize("drafts", [True, False])
def test_every_vocabulary(V, drafts):
    _same(_problem(V, [1, 5, 2, 0, 3, 1, 8], V, drafts))


@pytest.mark.parametrize("B,V", [(1, 131072), (76, 20000), (77, 20000), (152, 8192), (153, 9001), (304, 5000),
                                 (305, 5003), (700, 3001), (2000, 64)])
def test_every_cluster_size(B, V):
    _same(_problem(B, [1 + (i * 5) % 4 for i in range(B)], V))


def test_long_drafts():
    # more drafts than lanes, all accepted up to each place
    n = 80
    s = _problem(3, [n, n, n], 500)
    s["q"] = s["p"].clone()
    for r in range(3 * n - 1):
        s["tokens"][r + 1] = int(s["p"][r].argmax())
    s["u"].fill_(0.5)
    s["u"][n + 40] = 1.0                            # (u q < p fails: equal)
    s["u"][2 * n + 31] = 1.0
    _same(s)
    assert _run(s)[1].tolist() == [n, 41, 32]


def test_random_numbers_at_their_ends():
    s = _problem(4, [1, 1, 1, 3, 3, 3], 1000)
    s["w"] = torch.tensor([0.0, 1 - 2.0 ** -24, 0.5, 0.0, 1 - 2.0 ** -24, 0.25])
    s["u"][:] = torch.tensor([0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 1 - 2.0 ** -24, 1 - 2.0 ** -24, 0.1, 0.9, 0.9, 0.9])
    _same(s)
    s["p"][:, :600] = 0                             # the first token that weighs anything, not the first
    _same(s)
    s["p"][:, 700:] = 0
    _same(s)


def test_the_residual_decides():
    # the draft is worse everywhere but at two tokens: only they can be drawn
    V = 5000
    s = _problem(5, [2] * 40, V)
    p = torch.full((80, V), 1e-9)
    p[:, 17], p[:, 4000] = 0.3, 0.7
    q = torch.full((80, V), 2e-9)
    q[:, 17], q[:, 9] = 0.1, 0.9
    s["p"], s["q"] = p, q
    s["tokens"][:] = 9
    _same(s)
    assert set(_run(s)[0][:, 0].tolist()) <= {17, 4000}


def test_no_residual_draws_from_the_target_itself():
    s = _problem(6, [2, 2], 3000)
    s["q"] = s["p"] * 2                             # (not a distribution: nothing is left after the draft's share)
    s["u"].fill_(0.9)
    _same(s)


def test_nothing_to_draw_from():
    s = _problem(7, [1, 2], 300)
    s["p"].zero_()
    out, num = _run(s)
    assert num.tolist() == [1, 1] and (out == -1).all()
    _same(s)


def test_odd_values():
    # NaN and negative values count as 0; drafts outside the vocabulary are not accepted
    s = _problem(8, [3, 3, 3, 2], 4000)
    s["p"][0, :50] = float("nan")
    s["p"][1, 100:200] = -1.0
    s["q"][3, ::3] = float("nan")
    s["q"][4, ::5] = -2.0
    s["tokens"][7] = -1
    s["tokens"][10] = 4000
    _same(s)
    s["q"] = None
    _same(s)


def test_large_sums_and_small_ones():
    # weights of all sizes: tails of 1e-30 beside 1, and rows that sum to 1e-20 or 1e20
    s = _problem(9, [1] * 30, 20011, sharp=12.0)
    s["p"][10:20] *= 1e-20
    s["p"][20:] *= 1e20
    _same(s)


def test_strided_rows():
    V = 1001
    s = _problem(10, [2, 4, 1, 3], V)
    T = s["p"].shape[0]
    want = _run(s)
    wide = torch.full((2, T, V + 7), float("nan"), device="cuda")
    wide[0, :, 3:V + 3], wide[1, :, 3:V + 3] = s["p"].cuda(), s["q"].cuda()
    out = torch.full((4, 20), 99, dtype=torch.int32, device="cuda")
    num = torch.zeros(4, dtype=torch.int32, device="cuda")
    pb.verify_tokens(s["tokens"].cuda(), wide[0, :, 3:V + 3], torch.tensor(s["qsl"], dtype=torch.int32, device="cuda"),
                     s["u"].cuda(), s["w"].cuda(), out[:, :s["width"]], num, draft_probs=wide[1, :, 3:V + 3])
    assert torch.equal(out[:, :s["width"]].cpu(), want[0]) and torch.equal(num.cpu(), want[1])
    assert (out[:, s["width"]:] == 99).all()
    _same(s, want)


def test_requests_that_do_not_fit():
    s = _problem(11, [2, 5, 1], 400)
    scratch = torch.zeros(pb.SCRATCH_HEADER_BYTES, dtype=torch.uint8, device="cuda")
    out, num = _run(s, width=4, scratch=scratch)
    assert pb.check(scratch) == pb.DEVICE_CAPACITY
    assert (out[1] == 99).all() and num[1] == 99
    o, n = ref.verify(s["tokens"], s["p"], s["q"], s["qsl"], s["u"], s["w"], 5)
    assert torch.equal(out[[0, 2]], o[[0, 2], :4]) and torch.equal(num[[0, 2]], n[[0, 2]])


def test_replayed_graph_and_repeats():
    s = _problem(12, [1 + i % 5 for i in range(20)], 30000)
    B = 20
    d = {k: s[k].cuda() for k in ("tokens", "p", "q", "u", "w")}
    qsl = torch.tensor(s["qsl"], dtype=torch.int32, device="cuda")
    out = torch.zeros(B, s["width"], dtype=torch.int32, device="cuda")
    num = torch.zeros(B, dtype=torch.int32, device="cuda")
    call = lambda: pb.verify_tokens(d["tokens"], d["p"], qsl, d["u"], d["w"], out, num, draft_probs=d["q"])  # noqa: E731
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    t = _problem(13, [1 + i % 5 for i in range(20)], 30000)
    for k in d:
        d[k].copy_(t[k])
    g.replay()
    _same(t, (out.cpu(), num.cpu()))
