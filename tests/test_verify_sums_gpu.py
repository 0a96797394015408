"""The sums of pa_verify_tokens over the longest rows: the token that is drawn lies where the exact running sum crosses,
within 2^-36 of the whole (3000 times 2^-48, with every rounding of one sign)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from paged_kv_gqa_12_gb300 import binding as pb  # noqa: E402

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

UNIT = 2 ** 60                                       # all entries below are multiples of 1 / UNIT


def _whole(x):
    """float32 numbers times UNIT, as whole numbers."""
    m, e = np.frexp(np.asarray(x, np.float64))
    return [int(a * 2 ** 53) << (int(b) + 7) if b >= -7 else int(a * 2 ** 53) >> (-7 - int(b)) for a, b in zip(m, e)]


def _row(V, peaks, small, seed):
    """Entries of about `small`, some large ones in the first half, and, where the running sum passes `w` times the
    whole, 4096 entries of 2^-40: a sum that is off by 2^-31 of the whole would end up beside them."""
    rng = np.random.default_rng(seed)
    p = np.full(V, np.float32(small) * np.float32(1 / 3), np.float32)
    if seed % 2:
        p *= rng.random(V, np.float32) + np.float32(0.5)
    p[:V // 2:V // 16 if peaks else V] = np.float32(0.1)
    at = V // 2 + V // 16 + 5003
    p[at:at + 4096] = 2.0 ** -40
    # two entries before them bring the crossing to their middle: one of about 0.2, one of about 2^-22
    p[1000] = p[2000] = 0
    before, whole = sum(_whole(p[:at])), sum(_whole(p))
    w = np.float32((before / UNIT + 0.2) / (whole / UNIT + 0.2))
    wn = int(float(w) * 2 ** 24)
    need = (wn * whole - (before + 2048 * (UNIT >> 40)) * 2 ** 24) // (2 ** 24 - wn)       # x + y of them
    assert need > UNIT >> 10
    x = np.float32((need - (UNIT >> 22)) / UNIT)
    if x > need / UNIT:
        x = np.nextafter(x, np.float32(0))
    p[1000] = x
    p[2000] = np.float32((need - _whole([x])[0]) / UNIT)
    return p, w, at


def _draw(p, w, B):
    """The token of one request beside B - 1 that bring no row."""
    V = len(p)
    qsl = torch.ones(B + 1, dtype=torch.int32, device="cuda")
    qsl[0] = 0
    out = torch.full((B, 1), 99, dtype=torch.int32, device="cuda")
    num = torch.full((B,), 99, dtype=torch.int32, device="cuda")
    pb.verify_tokens(torch.zeros(1, dtype=torch.int32, device="cuda"), torch.from_numpy(p).cuda().view(1, V), qsl,
                     torch.zeros(1, device="cuda"), torch.full((B,), float(w), device="cuda"), out, num)
    assert num.tolist() == [1] + [0] * (B - 1) and (out[1:] == -1).all()
    return int(out[0])


@pytest.mark.parametrize("B", [1, 76, 153, 400])               # eight, four, two and one CTA a request
@pytest.mark.parametrize("peaks", [True, False])
@pytest.mark.parametrize("small", [2.0 ** -18, 2.0 ** -20, 2.0 ** -15])
@pytest.mark.parametrize("seed", [0, 1])
def test_the_crossing(B, peaks, small, seed):
    V = 1 << 20
    p, w, at = _row(V, peaks, small, seed)
    token = _draw(p, w, B)
    n = np.array(_whole(p), dtype=object)
    whole = int(n.sum())
    running = int(n[:token].sum())                   # without the token
    target = int(float(w) * 2 ** 24) * whole // 2 ** 24
    slack = whole >> 36
    assert at <= token < at + 4096
    assert running <= target + slack and running + int(n[token]) > target - slack, (token, at, (running - target) / whole)


@pytest.mark.parametrize("B", [1, 400])
@pytest.mark.parametrize("off", [0, 1])
def test_the_crossing_after_a_rejection(B, off):
    # rows that are not 16-byte aligned are summed another way; a rejected draft's entry is taken off
    V = 1 << 20
    p, w, at = _row(V, True, 2.0 ** -18, 0)
    x = 70000
    both = torch.zeros(2, V + 8)
    both[0, off:V + off] = torch.from_numpy(p)
    probs = both.cuda()[:, off:V + off]
    q = torch.zeros(2, V + 8)
    q[0, off + x] = 0.5                              # the draft: 0.5 of it, and it has less of the target
    qsl = torch.full((B + 1,), 2, dtype=torch.int32, device="cuda")
    qsl[0] = 0
    out = torch.full((B, 2), 99, dtype=torch.int32, device="cuda")
    num = torch.full((B,), 99, dtype=torch.int32, device="cuda")
    pb.verify_tokens(torch.tensor([0, x], dtype=torch.int32, device="cuda"), probs, qsl, torch.full((2,), 0.9, device="cuda"),
                     torch.full((B,), float(w), device="cuda"), out, num, draft_probs=q.cuda()[:, off:V + off])
    assert num.tolist() == [1] + [0] * (B - 1) and out[0, 1] == -1
    token = int(out[0, 0])
    n = np.array(_whole(p), dtype=object)
    n[x] = 0
    whole = int(n.sum())
    target = int(float(w) * 2 ** 24) * whole // 2 ** 24
    running = int(n[:token].sum())
    slack = whole >> 36
    assert running <= target + slack and running + int(n[token]) > target - slack, (token, at, (running - target) / whole)
