"""Random shapes of the 8-bit serving step against its 64-bit references: heads, groups, pages, ragged lengths and rows,
windows, sinks, caps, CTAs, scales of very different size."""
import random

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from paged_kv_gqa_12_gb300 import binding as pb  # noqa: E402
from tests import test_append_blocks_gpu as ap  # noqa: E402
from tests import test_block_attend_gpu as at  # noqa: E402
from tests import test_verify_tokens_gpu as vt  # noqa: E402


def _some(rng, n, lo, hi):
    return [rng.choice([lo, hi, rng.randint(lo, hi), rng.randint(lo, max(lo, hi // 10))]) for _ in range(n)]


@pytest.mark.parametrize("seed", range(24))
def test_attend(seed):
    rng = random.Random(seed)
    D, ps, Hkv = rng.choice([64, 128, 256]), rng.choice([16, 32, 64]), rng.choice([1, 2, 3, 4, 5, 8, 16])
    G = rng.choice([1, 2, 3, 4, 5, 8, 13]) if Hkv < 8 else rng.choice([1, 2, 4])
    B = rng.choice([1, 2, 7, 30])
    decode = rng.random() < 0.3
    most = 1 if decode else rng.choice([2, 3, 5, 9, 40, 150])
    B = 3 if most > 9 else B
    ctx = _some(rng, B, 0, rng.choice([10, 200, 1500]))
    new = [1] * B if decode else _some(rng, B, 0, most)
    new[0] = most
    s = at._problem(1000 + seed, rng.choice(["int8", "e4m3"]), G * Hkv, Hkv, D, ps, ctx, new,
                    window=rng.choice([0, 0, 1, 37, 300]), sinks=rng.random() < 0.4, cap=rng.choice([0.0, 0.0, 25.0]),
                    spread=rng.choice([1.0, 2.0, 100.0]))
    plan = at._plan(s, num_ctas=rng.choice([0, 0, 1, 2, 50, 700]),
                    host_seq_lens=s["seq"] if rng.random() < 0.5 else None)
    got = at._run(s, decode=decode, plan=plan)
    assert got[2] == 0
    at._close(got, at._want(s, decode=decode), (seed, D, ps, Hkv, G, ctx, new))


@pytest.mark.parametrize("seed", range(16))
def test_append(seed):
    rng = random.Random(seed)
    D, ps, Hkv, B = rng.choice([64, 128, 256]), rng.choice([16, 32, 64]), rng.choice([1, 2, 5, 8]), rng.choice([1, 3, 40])
    new = _some(rng, B, 0, rng.choice([1, 6, 90]))
    new[0] = max(new[0], 1)
    s = ap._problem(2000 + seed, rng.choice(["int8", "e4m3"]), Hkv, D, ps, _some(rng, B, 0, 100), new,
                    spread=rng.choice([1.0, 3.0, 50.0]))
    if rng.random() < 0.4:
        s["kv"] *= 2.0 ** rng.randint(-120, 100)
        s["k_scales"] *= 2.0 ** rng.randint(-20, 20)
    got, code = ap._run(s)
    assert code == 0
    ap._same(s, got)


@pytest.mark.parametrize("seed", range(16))
def test_verify(seed):
    rng = random.Random(seed)
    rows = _some(rng, rng.choice([1, 5, 60]), 0, rng.choice([1, 3, 8]))
    s = vt._problem(3000 + seed, rows, rng.choice([7, 300, 1024, 4097, 30011]), drafts=rng.random() < 0.6,
                    sharp=rng.choice([0.1, 2.0, 8.0]), near=rng.choice([1e-4, 0.3, 2.0]))
    if sum(rows):
        vt._same(s)
