"""The plan that kvq_attend_prompts makes in its workspace: an int32 count, and
from byte 256 on the items {begin, len, tok0, key tiles}."""
import numpy as np
import pytest

import serve_util as P
from gpu_util import Guarded, kb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kb()


def items(starts, total, group):
    """Those of the prompts in their order, of starts as they are."""
    tok = 2 * (128 // group)
    lo = np.clip(starts[:-1], 0, total)
    hi = np.maximum(np.minimum(starts[1:], total), lo)
    res = [(a, z - a, t, -(-min(t + tok, z - a) // 128)) for a, z in zip(lo, hi) for t in range(0, z - a, tok)]
    return res, total // tok + min(len(starts) - 1, total)


CASES = {
    "overlapping": ([0, 600] * 400 + [0], 600, 64),
    "overlapping, more than a pass": ([0, 600] * 1000 + [0], 600, 64),
    "overlapping from the second pass on": ([0] * 1100 + [0, 600] * 700 + [5], 600, 64),
    "out of order, none too many": ([0, 90, 80, 400, 380, 600, 0], 600, 32),
    "in order": (list(range(0, 600, 7)), 600, 64),
}


@pytest.mark.parametrize("name", CASES)
def test_no_more_items_than_the_workspace_holds(b, name):
    """The first in the prompts' order, each once, those of many key tiles first; nothing outside is written."""
    import torch
    starts, total, G = CASES[name]
    starts, Hk, C = np.array(starts, np.int64), 4, 64
    n = len(starts) - 1
    x = P.upload_bf16(P.packed(np.random.default_rng(4), total, (G + 2) * Hk, C))
    q, k, v = (t.contiguous() for t in x.split([Hk * G, Hk, Hk], 1))
    g = Guarded()
    out = g.alloc(total * Hk * G * C * 2).view(torch.bfloat16).view(total, Hk * G, C)
    lse = g.alloc(total * Hk * G * 4).view(torch.float32).view(total, Hk * G)
    wB = b.kvq_attend_prompts_workspace(n, total, G, Hk, C)
    ws = g.alloc(wB)
    b.attend_prompts(q, k, v, torch.from_numpy(starts.astype(np.int32)).cuda(), out, lse, ws)
    g.check(name)
    want, most = items(starts, total, G)
    assert wB == 256 + 16 * most
    want = want[:most]
    count = int(ws[:4].view(torch.int32))
    got = [tuple(r) for r in ws[256:256 + 16 * count].view(torch.int32).view(-1, 4).tolist()]
    assert count == len(want) and sorted(got) == sorted(want)
    keys = [r[3] for r in got]
    assert keys == sorted(keys, reverse=True)
    assert b.kvq_wait_timeouts() == 0
