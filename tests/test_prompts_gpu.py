"""kvq_attend_prompts against the formula in binary64.

Tolerances (u = 2^-8, the largest relative error of a rounding to bf16; e twice
the logits' error, stream_util.logit_error; L the prompt's length):
  lse: e + (L + 64) 2^-23 + 4 2^-23 (|lse| + 1)
  out: (u + e + (L + 64) 2^-23) sum_t p_t |v_t| + u |out|
"""
import zlib

import numpy as np
import pytest

import serve_util as P
import stream_util as S
from gpu_util import Guarded, kb

pytestmark = pytest.mark.gpu
SENTINEL = 0x1234                                # bf16 bits of rows that no call may write


@pytest.fixture(scope="module")
def b():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kb()


#  lens, kv_heads, group, C, extras: rows before the first and behind the last prompt, fused, scale of q
CASES = {
    "one token": ([1], 1, 1, 128, {}),
    "one token, C 64": ([1], 2, 3, 64, {}),
    "tokens alone": ([1] * 9, 2, 4, 128, {}),
    "17 tokens": ([17], 8, 4, 128, dict(fused=True)),
    "a tile of rows": ([32], 1, 4, 128, {}),
    "a tile of rows and one": ([33], 1, 4, 128, {}),
    "two tiles and one": ([65], 2, 4, 64, {}),
    "127, 128, 129": ([127, 128, 129], 1, 1, 128, {}),
    "255, 256, 257": ([255, 256, 257], 1, 1, 64, {}),
    "ragged": ([3, 700, 1, 64, 250, 511, 2, 90], 2, 4, 128, dict(fused=True)),
    "ragged, C 64": ([300, 1, 129, 31], 3, 2, 64, dict(fused=True)),
    "empty prompts": ([0, 5, 0, 0, 130, 0], 1, 8, 128, {}),
    "all empty": ([0, 0], 1, 4, 128, dict(behind=3)),
    "no tokens": ([0, 0], 2, 4, 128, {}),
    "rows outside": ([40, 150], 2, 4, 128, dict(before=7, behind=140)),
    "group of 3": ([100, 43, 200], 2, 3, 128, {}),
    "group of 5": ([100, 27], 1, 5, 64, {}),
    "group of 7": ([75, 300], 2, 7, 128, dict(fused=True)),
    "group of 12": ([140], 1, 12, 128, {}),
    "group of 43": ([33], 1, 43, 64, {}),
    "group of 64": ([50, 9], 1, 64, 128, {}),
    "many heads": ([70, 20], 40, 1, 64, {}),
    "one head": ([700], 1, 1, 128, {}),
    "loud": ([150, 60], 1, 4, 128, dict(scale=6.0)),
    "long": ([1500], 1, 2, 128, {}),
    "long, C 64": ([1111, 400], 1, 3, 64, {}),
    "many prompts": ([(i * 37) % 50 for i in range(300)], 1, 2, 64, {}),
    # more pairs than SMs, so that a plan is made: prompts whose items a warp shares, and last items of one row tile
    "planned": ([1400, 300, 77], 4, 8, 64, {}),
    "planned, C 128": ([900, 40, 513], 3, 8, 128, dict(fused=True)),
    "planned, one query head": ([700, 515, 5], 40, 1, 128, {}),
    "many pairs of one row tile a CTA": ([1 + i % 7 for i in range(900)], 3, 2, 64, {}),
    "many pairs of two row tiles a CTA": ([129 + i % 7 for i in range(260)], 5, 1, 64, {}),
    "lone last row tiles": ([1100, 1030, 260], 2, 1, 128, {}),
    "lone last row tiles, C 64": ([770, 1030], 2, 2, 64, {}),
    "more prompts than a pass of the plan": ([i % 3 for i in range(1500)], 1, 1, 64, {}),
    "planned, rows outside": ([333, 0, 500, 1], 8, 8, 64, dict(before=3, behind=50)),
}


def build(name):
    rng = np.random.default_rng(zlib.crc32(name.encode()))
    lens, Hk, G, C, ex = CASES[name]
    total = ex.get("before", 0) + sum(lens) + ex.get("behind", 0)
    x = P.packed(rng, total, (G + 2) * Hk, C, scale=1.0)
    if "scale" in ex:
        x[:, :G * Hk] = P.packed(rng, total, G * Hk, C, scale=ex["scale"])
    return lens, Hk, G, C, ex, x, P.starts_of(lens, ex.get("before", 0))


def views(x, Hk, G, fused):
    t = P.upload_bf16(x)
    q, k, v = t.split([Hk * G, Hk, Hk], 1)
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def check(name, out, lse, x, starts, Hk, G):
    """out and lse (host, binary64) against the prompts' formula."""
    rows = S.bf16_to_f64(x)
    for s in range(len(starts) - 1):
        a, z = starts[s], starts[s + 1]
        if a == z:
            continue
        q, k, v = np.split(rows[a:z], [Hk * G, Hk * G + Hk], 1)
        wl, wo, wa, e = P.prompt_reference(q, k, v, G)
        tl, to = P.tolerances(wl, wo, wa, e, z - a)
        P.close(lse[a:z], wl, tl, f"{name}: lse of prompt {s}")
        P.close(out[a:z], wo, to, f"{name}: out of prompt {s}")


@pytest.mark.parametrize("name", CASES)
def test_attend_prompts(b, name):
    import torch
    lens, Hk, G, C, ex, x, starts = build(name)
    total, H = x.shape[0], Hk * G
    q, k, v = views(x, Hk, G, ex.get("fused", False))
    g = Guarded()
    out = g.alloc(max(total * H * C * 2, 16)).view(torch.bfloat16)[:total * H * C].view(total, H, C)
    lse = g.alloc(max(total * H * 4, 16)).view(torch.float32)[:total * H].view(total, H)
    out.view(torch.int16).fill_(SENTINEL)
    lse.fill_(-7.0)
    ws = g.alloc(max(b.kvq_attend_prompts_workspace(len(lens), total, G, Hk, C), 16))
    b.attend_prompts(q, k, v, torch.from_numpy(starts).cuda(), out, lse, ws)
    g.check(name)
    bits, gl = out.view(torch.int16).cpu().numpy(), P.f64(lse)
    check(name, P.f64(out), gl, x, starts, Hk, G)
    for s in (slice(0, starts[0]), slice(starts[-1], total)):
        assert (bits[s] == SENTINEL).all() and (gl[s] == -7.0).all(), "rows of tokens in no prompt were written"
    assert b.kvq_wait_timeouts() == 0


def test_default_arguments_and_equal_bits(b):
    import torch
    lens, Hk, G, C, _, x, starts = build("ragged")
    q, k, v = views(x, Hk, G, True)
    st = torch.from_numpy(starts).cuda()
    one = b.attend_prompts(q, k, v, st)
    two = b.attend_prompts(q.contiguous(), k, v.contiguous(), st)
    for a, c in zip(one, two):
        assert torch.equal(a, c)
    qc = q.contiguous()
    b.attend_prompts(qc, k, v, st, out=qc)                             # in place
    assert torch.equal(qc, one[0])


def test_nothing_to_do(b):
    import torch
    e = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    out, lse = b.attend_prompts(e, e[:, :2], e[:, 2:], torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4)
    x = torch.zeros((5, 4, 128), dtype=torch.bfloat16, device="cuda")
    y, z = x.clone(), torch.full((5, 4), 3.0, device="cuda")
    b.attend_prompts(x, x[:, :2].contiguous(), x[:, 2:].contiguous(), torch.zeros(1, dtype=torch.int32, device="cuda"), y, z)
    assert torch.equal(y, x) and (z == 3.0).all()


@pytest.mark.parametrize("starts", [[-5, 40, 1000], [30, 10, 60], [0, 2**31 - 1], [-2**31, 2**31 - 1], [60, 0]])
def test_starts_out_of_order_or_range_stay_inside(b, starts):
    """The results are unspecified; nothing outside of the tensors is touched, and every wait ends."""
    import torch
    rng = np.random.default_rng(5)
    total, Hk, G, C = 60, 2, 4, 128
    q, k, v = views(P.packed(rng, total, (G + 2) * Hk, C), Hk, G, False)
    g = Guarded()
    out = g.alloc(total * Hk * G * C * 2).view(torch.bfloat16).view(total, Hk * G, C)
    lse = g.alloc(total * Hk * G * 4).view(torch.float32).view(total, Hk * G)
    st = torch.tensor(starts, dtype=torch.int64).to(torch.int32).cuda()
    b.attend_prompts(q, k, v, st, out, lse, g.alloc(max(b.kvq_attend_prompts_workspace(len(starts) - 1, total, G, Hk, C), 16)))
    g.check("starts")
    assert b.kvq_wait_timeouts() == 0


def test_captured_calls_replay_with_other_lengths(b):
    """Two captured graphs, each with a workspace of its own, on the lengths that starts holds at the replay."""
    import torch
    rng = np.random.default_rng(6)
    Hk, G, C, total = 2, 4, 128, 640
    x = P.packed(rng, total, (G + 2) * Hk, C)
    q, k, v = views(x, Hk, G, True)
    sets = [[640, 0, 0, 0], [1, 300, 2, 337], [160, 160, 160, 160], [0, 0, 639, 0]]
    sts = [torch.from_numpy(P.starts_of(sets[0])).cuda() for _ in range(2)]
    outs = [(torch.empty((total, Hk * G, C), dtype=torch.bfloat16, device="cuda"),
             torch.empty((total, Hk * G), device="cuda")) for _ in range(2)]
    wB = b.kvq_attend_prompts_workspace(4, total, G, Hk, C)
    wss = [torch.empty(max(wB, 16), dtype=torch.uint8, device="cuda") for _ in range(2)]
    b.attend_prompts(q, k, v, sts[0], *outs[0], wss[0])
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            b.attend_prompts(q, k, v, sts[i], *outs[i], wss[i])
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for lens in sets:
        for i in range(2):
            sts[i].copy_(torch.from_numpy(P.starts_of(lens if i == 0 else lens[::-1])))
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            check("replay", P.f64(outs[i][0]), P.f64(outs[i][1]), x, P.starts_of(lens if i == 0 else lens[::-1]), Hk, G)


def test_on_another_stream(b):
    import torch
    lens, Hk, G, C, _, x, starts = build("group of 7")
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        q, k, v = views(x, Hk, G, False)
        dev = torch.from_numpy(starts).cuda()
    out, lse = b.attend_prompts(q, k, v, dev, stream=st)
    st.synchronize()
    check("stream", P.f64(out), P.f64(lse), x, starts, Hk, G)


NAN, INF, NEG = np.uint16(0x7FC0), np.uint16(0x7F80), np.uint16(0xFF80)


@pytest.mark.parametrize("shape", [([130, 60, 257], 2, 4, 128), ([700, 33], 1, 2, 64), ([40, 9], 1, 3, 128)])
def test_values_and_keys_that_are_not_finite(b, shape):
    """A value reaches its channel of the rows of its own prompt that see its token, and no other; a logit of NaN makes
    NaN of the rows that see it; both leave every other row what it is without them."""
    import torch
    lens, Hk, G, C = shape
    rng = np.random.default_rng(sum(lens))
    starts = P.starts_of(lens)
    total, H = sum(lens), Hk * G
    x = P.packed(rng, total, H + 2 * Hk, C)
    clean = x.copy()
    V = x[:, H + Hk:]
    V[starts[0] + 20, 0, 5] = INF
    V[starts[0] + 35, 0, 5] = NEG                # with the one before: NaN
    V[starts[0] + 36, 0, 7] = NEG
    V[starts[1] - 1, 0, 9] = NAN                 # the last token of a prompt: no other prompt sees it
    V[starts[1], 0, 11] = INF                    # the first of the next
    V[total - 1, Hk - 1, C - 1] = NAN
    K = x[:, H:H + Hk]
    K[starts[1] + 4, Hk - 1, 3] = NAN
    q, k, v = views(x, Hk, G, True)
    out, lse = (P.f64(t) for t in b.attend_prompts(q, k, v, torch.from_numpy(starts).cuda()))
    rows = S.bf16_to_f64(clean)
    for s in range(len(lens)):
        a, z = starts[s], starts[s + 1]
        qs, ks, vs = np.split(rows[a:z], [H, H + Hk], 1)
        wl, wo, wa, e = P.prompt_reference(qs, ks, vs, G)
        tl, to = P.tolerances(wl, wo, wa, e, z - a)
        odd = S.bf16_to_f64(V[a:z])
        for h in range(Hk):
            hs = slice(h * G, (h + 1) * G)
            for c in np.unique(np.argwhere(~np.isfinite(odd[:, h]))[:, 1]):
                seen = np.where(np.isfinite(odd[:, h, c]), 0.0, odd[:, h, c])
                with np.errstate(invalid="ignore"):
                    add = np.cumsum(seen)
                wo[:, hs, c] += add[:, None]
                to[~np.isfinite(add), hs, c] = 0.0
            nan = np.argwhere(np.isnan(S.bf16_to_f64(K[a:z, h])).any(-1))
            if len(nan):
                wo[nan[0, 0]:, hs] = np.nan
                wl[nan[0, 0]:, hs] = np.nan
        P.close(lse[a:z], wl, tl, f"lse of prompt {s}")
        P.close(out[a:z], wo, to, f"out of prompt {s}")


def test_logits_of_infinity(b):
    """-inf alone: a row that sees nothing; +inf: NaN."""
    import torch
    one = torch.zeros((3, 1, 64), dtype=torch.bfloat16, device="cuda")
    q, k, v = one.clone(), one.clone(), one.clone()
    q[:, 0, 0], k[0, 0, 0], k[1, 0, 0], v[:, 0, 1] = 1.0, -float("inf"), -float("inf"), 2.0
    st = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    out, lse = b.attend_prompts(q, k, v, st)
    assert out[0].abs().sum() == 0 and out[1].abs().sum() == 0 and (lse[:2] == -float("inf")).all()
    assert out[2, 0, 1] == 2.0 and abs(float(lse[2])) < 1e-6
    k[1, 0, 0] = float("inf")
    out, lse = b.attend_prompts(q, k, v, st)
    assert out[0].abs().sum() == 0 and out[1:].isnan().all() and lse[1:].isnan().all()
