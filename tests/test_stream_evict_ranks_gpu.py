"""kvq_evict_blocks: the order of blocks whose scores are equal or nearly equal sums
of long rows.

Blocks are ranked by the sum of their scores.  Sums of the same numbers in
another order are equal, so the earlier block stays; the sums here span at most
63 bits, which the kernel adds without an error.
"""
from fractions import Fraction

import numpy as np
import pytest

from gpu_util import kb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kb()


def ranked(b, sc, block, budget):
    """The kept blocks of a store of small per-token groups, by the GPU."""
    import torch
    outer, T = sc.shape
    qp = b.QParams.sym(8, axis=b.ALONG_C, group=0, scale_dtype=b.F32)
    kv = [tuple(torch.zeros(n, dtype=torch.uint8, device="cuda") for n in b.kvq_quantized_sizes((outer, T, 8), b.BF16, qp)[:2])
          + (None, None) for _ in range(2)]
    cache = b.KVCache(k=kv[0], v=kv[1], shape=(outer, T, 8), kqp=qp, vqp=qp, tq=T, nres=0, resid_rows=0)
    return b.evict_blocks(cache, torch.from_numpy(sc).cuda(), budget, 0, block)[2].cpu().numpy()


def span_bits(row):
    """bits between the top of the row's sum and the last bit of its smallest number"""
    m, e = np.frexp(row[row != 0].astype(np.float64))
    return int(np.ceil(np.log2(np.abs(row).astype(np.float64).sum()))) - (int(e.min()) - 24)


@pytest.mark.parametrize("block", [64, 128, 1024, 4096])
@pytest.mark.parametrize("signs", [False, True])
def test_permuted_blocks_tie(b, block, signs):
    """Block 2 i + 1 holds block 2 i's scores in another order: of every pair the first one stays."""
    rng = np.random.default_rng(block + signs)
    pairs, outer = 48, 4
    a = np.exp(2.5 * rng.standard_normal((outer, pairs, block))).astype(np.float32)
    if signs:
        a *= rng.choice([-1.0, 1.0], a.shape).astype(np.float32)
    assert max(span_bits(r) for r in a.reshape(-1, block)) <= 63
    sc = np.stack([a, np.stack([[rng.permutation(r) for r in s] for s in a])], 2).astype(np.float32)
    sc = sc.reshape(outer, 2 * pairs * block)
    for budget in (1, 7, 2 * pairs - 3):                 # odd: a pair is cut
        keep = ranked(b, sc, block, budget)
        for o in range(outer):
            s = [sum(map(Fraction, map(float, sc[o, i * block:(i + 1) * block])), Fraction(0)) for i in range(0, 2 * pairs, 2)]
            s = [x for x in s for _ in range(2)]
            want = sorted(sorted(range(2 * pairs), key=lambda i: (-s[i], i))[:budget])
            assert keep[o].tolist() == want


def test_long_blocks_are_told_apart(b):
    """Sums of 2^18 positive scores that differ by one part in 2^40: the larger stays."""
    rng = np.random.default_rng(3)
    block = 1 << 18
    a = rng.random((4, block)).astype(np.float32) + 0.5
    sc = np.concatenate([a, a[:, rng.permutation(block)]], 1)
    for o in range(4):                                   # one small number more in the later block
        sc[o, o] = 0.0
        sc[o, block + int(np.flatnonzero(sc[o, block:] == a[o, o])[0])] = np.float32(2.0 ** -22)
        exact = [sum(map(Fraction, map(float, sc[o, i * block:(i + 1) * block])), Fraction(0)) for i in range(2)]
        assert 0 < exact[1] - exact[0] < exact[0] / (1 << 39)
    assert ranked(b, sc, block, 1).ravel().tolist() == [1] * 4


@pytest.mark.parametrize("extra", [0, 1])
def test_equal_parts_of_an_infinite_or_overflowing_sum(b, extra):
    """Sums beyond float32 are infinities and tie; NaN ranks last."""
    block = 64
    big = np.full(block, 3e38, np.float32)
    rows = [big, np.full(block, 1.0, np.float32), big.copy(), -big, np.full(block, np.nan, np.float32),
            np.where(np.arange(block) == 7, np.inf, 2.0).astype(np.float32)]
    sc = np.concatenate(rows)[None]
    order = [0, 2, 5, 1, 3, 4]
    for budget in range(1, 6):
        assert ranked(b, sc, block, budget)[0].tolist() == sorted(order[:budget])
