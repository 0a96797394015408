"""NaN among an e4m3 cache's V codes reaches the rows that attend to its key, in its dimension, and no other value: a
later token of the same request, or one that has left the window, stays masked."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests import test_block_attend_gpu as at  # noqa: E402


def _same(got, want):
    o, l, to, tl = want
    out, lse = got[0].double(), got[1].double()
    nan = o.isnan()
    assert torch.equal(out.isnan(), nan), ((out.isnan() != nan).nonzero()[:5], int(nan.sum()))
    assert ((out - o).abs() <= to)[~nan].all()
    assert ((lse - l).abs() <= tl).all()
    return int(nan.sum())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [[4, 1, 2, 3], [2, 2, 2, 2], [5, 12, 9, 1], [70, 33, 90, 1]])
@pytest.mark.parametrize("opts", [dict(), dict(window=3, sinks=True), dict(window=40, cap=20.0)])
@pytest.mark.parametrize("ps", [16, 64])
def test_later_tokens_and_tokens_before_the_window(D, new, opts, ps):
    g = torch.Generator().manual_seed(D + ps)
    ctx = [100, 0, 15, 700]
    s = at._problem(31 + D, "e4m3", 8, 2, D, ps, ctx, new, dirty=False, **opts)
    seen = 0
    W = opts.get("window", 0)
    for b, n in enumerate(new):
        # some of the new tokens and some just before the window: one dimension of one head each, of either sign
        at_keys = set(torch.randint(ctx[b], ctx[b] + n, (3,), generator=g).tolist())
        if W:
            at_keys |= {max(0, ctx[b] - W + int(i)) for i in torch.randint(0, n + 2, (2,), generator=g)}
        for j in at_keys:
            if j >= s["seq"][b]:
                continue
            page, h = int(s["table"][b, j // ps]), int(torch.randint(0, 2, (1,), generator=g))
            d = int(torch.randint(0, D, (1,), generator=g))
            s["v_cache"][page, j % ps, h, d] = 0x7f if d % 2 else 0xff
    for kw in (dict(), dict(num_ctas=1), dict(num_ctas=50)):
        plan = at._plan(s, **kw)
        got = at._run(s, plan=plan)
        assert got[2] == 0
        seen += _same(got, at._want(s))
    assert seen > 0


@pytest.mark.parametrize("new", [[3, 4], [70, 80]])
def test_codes_of_minus_zero_are_zeros(new):
    s = at._problem(5, "e4m3", 8, 2, 64, 16, [50, 3], new)
    g = torch.Generator().manual_seed(1)
    zero = torch.rand(s["v_cache"].shape, generator=g) < 0.3
    s["v_cache"][zero] = 0x80
    got = at._run(s)
    at._close(got, at._want(s))


@pytest.mark.parametrize("new", [[4, 2], [70, 80]])
def test_a_token_of_nan_and_its_own_row_alone(new):
    # the last token's V is NaN everywhere: all other rows are as without it
    s = at._problem(6, "e4m3", 8, 2, 128, 16, [300, 20], new)
    for b, L in enumerate(s["seq"]):
        s["v_cache"][int(s["table"][b, (L - 1) // 16]), (L - 1) % 16] = 0x7f
    got = at._run(s)
    rows = torch.zeros(s["q"].shape[0], dtype=torch.bool)
    rows[[s["qsl"][1] - 1, s["qsl"][2] - 1]] = True
    assert got[0][rows].isnan().all() and got[0][~rows].isfinite().all()
    _same(got, at._want(s))
