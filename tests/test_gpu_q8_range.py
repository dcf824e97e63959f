"""The 8-bit cache's calls at the ends of their ranges: scores, scales, queries and log sums
far from 1, weights too small for the 16 bits they are held in.

Tolerances are those of test_gpu_q8.py (a score is off by dS, a weight by a factor
1 + rel), widened where a test says so:

* A weight times its token's V scale is held in fp16 with the row's largest at 2^6 or more:
  below 2^-20 of the largest it is subnormal there, off by at most half a step, 2^-25, or
  2^-31 of the largest.
* In the kernel for chunks of queries a query element is two E4M3 parts, the row's largest
  in [2^7, 2^8).  An element of exponent e has 8 bits down to 2^(e-7): the first part leaves a
  multiple of that, at most 8 of them, which the second part holds if the steps it has at its
  smallest, 2^-9, reach: e >= -2, elements down to 2^-9 of the power of two below the row's
  largest.  Those below are off by half a step, 2^-10, at most 2^-17 of the row's largest.
"""
import numpy as np
import pytest

from oracle import q8cache as q8
from tests.test_gpu_q8 import _dt, attend, check_attend, check_mass, filled, head_values, host_codes, poisoned

pytestmark = pytest.mark.gpu

# every kernel: few rows, 16-row tiles (one and several), chunks (a lone tile, a pair), f32
KERNELS = [("bf16", 1), ("bf16", 8), ("bf16", 12), ("bf16", 40), ("bf16", 100), ("bf16", 300), ("f32", 1), ("f32", 5)]


def attend_one_head(c, h, Q, rows=None):
    """(q, O, lse, size) of head h in fp64 (rows: those of them)."""
    q = Q[h, slice(None) if rows is None else rows].double().cpu().numpy()
    K, V = head_values(c, h)
    sc = 1.0 / np.sqrt(Q.shape[2])
    dS = (np.abs(q) @ np.abs(K).T).max(1, keepdims=True) * sc * 2.0 ** -17
    return (*q8.attend(q, K, V, sc), dS)


def check_rows(O, lse, ref, rows, dt, lost=0.0, dS_more=0.0):
    """One head's outputs against attend_one_head's; `lost`: what else they may be off by, `dS_more`:
    what else a score may be."""
    import torch
    want, want_lse, size, dS = ref
    dS = dS + dS_more
    pick = slice(None) if rows is None else rows
    half = torch.finfo(dt).eps / 2
    rel = 4 * dS + 2.0 ** -11 + 2.0 ** -18
    tol = rel * size + lost
    tol = tol + half * (np.abs(want) + tol)
    err = np.abs(O[pick].double().cpu().numpy() - want)
    assert np.all(err <= tol), float((err / tol).max())
    if lse is not None:
        el = np.abs(lse[pick].double().cpu().numpy() - want_lse)
        tl = dS[:, 0] + 2.0 ** -18 + 2.0 ** -17 * (1 + np.abs(want_lse))
        assert np.all(el <= tl), float((el / tl).max())


# ------------------------------------------------------------------ weights
@pytest.mark.parametrize("dtype,rows", KERNELS)
@pytest.mark.parametrize("below", [60.0, 80.0, 200.0])
def test_mass_of_log_sums_far_below_the_scores(below, dtype, rows):
    """A caller's lse (of another part of the cache, say) may lie far below the scores: weights
    are then large, infinite where they pass fp32's range, and never negative."""
    import torch
    torch.manual_seed(rows)
    c = filled(3, 128, 512, 64, dtype, [500, 129, 1], rows, max_queries=rows)
    Q = (2 * torch.randn(3, rows, 128, device="cuda")).to(_dt(dtype)[0])
    _, lse = attend(c, Q)
    lse -= below
    prev = c.mass.clone()
    c.accumulate(Q, lse, decay=0.5)
    assert c.status() == 0
    if below < 88:                         # every weight is in range, and their sums by e^3 at least
        check_mass(c, Q, lse, 0.5, prev)
        return
    for h in range(3):
        n = int(c.len[h])
        K, _ = head_values(c, h)
        q, z = Q[h].double().cpu().numpy(), lse[h].double().cpu().numpy()
        got = c.mass[h, :n].double().cpu().numpy()
        ref = q8.mass(q, K, 128 ** -0.5, z)
        s = (np.abs(q) @ np.abs(K).T).max() * 128 ** -0.5
        rel = 2 * s * 2.0 ** -17 + 2.0 ** -18 + 2.0 ** -22 * (s + np.abs(z).max()) + 2.0 ** -20
        sure = ref > 2.0 ** 128 * (1 + rel)
        assert n == 1 or sure.any()
        assert np.all(np.isposinf(got[sure]))
        fine = ref < 2.0 ** 128 * (1 - 2 * rel)
        assert np.all(np.abs(got[fine] - ref[fine]) <= rel * ref[fine] + 2.0)


@pytest.mark.parametrize("dtype,rows", KERNELS)
def test_mass_of_the_lowest_log_sums(dtype, rows):
    """lse of the type's lowest value is a number, not -inf: weights pass fp32's range; beside
    rows of -inf, which weigh nothing."""
    import torch
    torch.manual_seed(rows)
    c = filled(2, 64, 512, 64, dtype, [500, 130], rows, max_queries=rows)
    Q = torch.randn(2, rows, 64, device="cuda").to(_dt(dtype)[0])
    lse = torch.full((2, rows), float("-inf"), device="cuda")
    prev = c.mass.clone()
    for at in {0, rows // 2, rows - 1}:
        for low in (-1e30, torch.finfo(torch.float32).min):
            lse[0, at] = low
            c.accumulate(Q, lse, prev=prev)
            assert bool(torch.isposinf(c.mass[0, :500]).all())
            assert torch.equal(c.mass[1, :130], prev[1, :130])
        lse[0, at] = float("-inf")


@pytest.mark.parametrize("dtype,rows", KERNELS)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -3e38])
def test_mass_of_padded_rows(value, dtype, rows):
    """Rows of lse -inf weigh nothing, whatever their queries hold: what the others give alone."""
    import torch
    torch.manual_seed(rows)
    c = filled(2, 128, 512, 64, dtype, [500, 77], rows, max_queries=rows)
    Q = torch.randn(2, rows, 128, device="cuda").to(_dt(dtype)[0])
    _, lse = attend(c, Q)
    pad = torch.rand(2, rows, device="cuda") < 0.5
    pad[0, rows // 2] = True
    pad[1, 0] = False
    lse[pad] = float("-inf")
    prev = c.mass.clone()
    Q[pad] = 0
    c.accumulate(Q, lse, prev=prev)
    want = c.mass.clone()
    c.mass.copy_(prev)
    Q[pad] = value
    c.accumulate(Q, lse, prev=prev)
    assert c.status() == 0
    assert torch.equal(c.mass.view(torch.int32), want.view(torch.int32))
    check_mass(c, torch.where(pad[..., None], torch.zeros_like(Q), Q), lse, 1.0, prev)


# ------------------------------------------------------------------ scores
@pytest.mark.parametrize("dtype,rows", KERNELS + [("bf16", 70)])
@pytest.mark.parametrize("n", [40, 30000])
def test_attend_every_score_past_the_range_of_floats(n, dtype, rows):
    """Scores below -2^128 count as -inf.  Rows with no other see nothing: zeros and lse -inf,
    whole or cut into pieces; rows of the other head are untouched."""
    import torch
    torch.manual_seed(rows)
    dt, cap = _dt(dtype)[0], -(-n // 64) * 64
    c = filled(2, 128, cap, 64, dtype, [n, n - 7], 3, max_queries=rows)
    lo = -2.0 ** 126
    c.K[0, :n] = 0
    c.K[0, :n, 0] = torch.tensor([lo * 2.0 ** -119]).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    c.k_scale[0, :-(-n // 64)] = 2.0 ** 119
    Q = torch.randn(2, rows, 128, device="cuda").to(dt)
    Q[0, :, 0] = 64.0
    O, lse = attend(c, Q)
    assert c.status() == 0
    assert bool((O[0] == 0).all()) and bool(torch.isneginf(lse[0]).all())
    pick = None if n < 100 else np.array([0, rows - 1])
    K, V = head_values(c, 1)
    assert np.isfinite(K).all()
    ref = attend_one_head(c, 1, Q, pick)
    check_rows(O[1], lse[1], ref, pick, dt)


@pytest.mark.parametrize("dtype,rows", KERNELS)
def test_attend_infinite_queries_against_one_sign(dtype, rows):
    """An infinite element gives a NaN row also where it would send every score to -inf."""
    import torch
    torch.manual_seed(rows)
    dt = _dt(dtype)[0]
    c = filled(1, 64, 256, 32, dtype, [200], 4, max_queries=rows)
    c.K[0, :200, 9] = torch.tensor([-2.0]).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    Q = torch.randn(1, rows, 64, device="cuda").to(dt)
    clean, clean_lse = attend(c, Q)
    at = rows // 2
    Q[0, at, 9] = float("inf")
    O, lse = attend(c, Q)
    assert bool(O[0, at].isnan().all()) and bool(lse[0, at].isnan())
    keep = torch.arange(rows, device="cuda") != at
    assert torch.equal(O[0, keep], clean[0, keep]) and torch.equal(lse[0, keep], clean_lse[0, keep])


# ------------------------------------------------------------------ V scales
@pytest.mark.parametrize("dtype,rows", KERNELS)
@pytest.mark.parametrize("exp", [-122, -100, 100])
def test_attend_scales_of_any_size(exp, dtype, rows):
    """V scales far from 1, also below the smallest that an append writes."""
    import torch
    torch.manual_seed(rows)
    c = filled(2, 128, 512, 16, dtype, [500, 77], 2, max_queries=rows)
    c.v_scale *= 2.0 ** (exp + 6)
    Q = (2 * torch.randn(2, rows, 128, device="cuda")).to(_dt(dtype)[0])
    O, lse = attend(c, Q)
    assert c.status() == 0
    check_attend(c, Q, O, lse)


@pytest.mark.parametrize("dtype,rows", KERNELS)
@pytest.mark.parametrize("first", [True, False])
def test_attend_blocks_of_zeros_among_others(first, dtype, rows):
    """Zero blocks as an append writes them (scale 2^-100) at the head's start or behind others:
    their tokens weigh as much as the rest."""
    import torch
    torch.manual_seed(rows)
    n, dt = 500, _dt(dtype)[0]
    c = poisoned(2, 64, 512, 16, dtype, max_queries=rows)
    K, V = torch.randn(2, 2, n, 64, device="cuda")
    zero = (torch.arange(n, device="cuda") // 16) % 2 == (0 if first else 1)
    V[0, zero] = 0
    V[1, zero] = 0
    V[1] *= 2.0 ** 6                        # scales 2^100 apart
    c.append(K.to(dt), V.to(dt))
    assert float(c.v_scale[0, 0 if first else 1]) == 2.0 ** -100
    Q = torch.randn(2, rows, 64, device="cuda").to(dt)
    O, lse = attend(c, Q)
    check_attend(c, Q, O, lse)


@pytest.mark.parametrize("dtype,rows", [("bf16", 1), ("bf16", 12), ("bf16", 60), ("bf16", 140), ("f32", 2)])
def test_attend_millions_of_zeros(dtype, rows):
    """A head of zeros, as appended, has a finite lse: 2^22 + 5 tokens."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    n = (1 << 22) + 5
    c = kvb.Q8Cache(1, 64, n + 59, 64, dtype=_dt(dtype)[1], max_queries=rows)
    c.K.zero_()
    c.V.zero_()
    c.k_scale.fill_(2.0 ** -100)
    c.v_scale.fill_(2.0 ** -100)
    c.len.fill_(n)
    Q = torch.randn(1, rows, 64, device="cuda").to(_dt(dtype)[0])
    O, lse = attend(c, Q)
    assert c.status() == 0
    assert bool((O == 0).all())
    # a sum of up to 2000 equal terms a lane, 200 sums merged: 2200 roundings of 2^-24 at most, and
    # the roundings of a log sum put together from terms of about 100: 2^-16
    assert float((lse.double() - np.log(n)).abs().max()) <= 2200 * 2.0 ** -24 + 2.0 ** -15


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_of_nothing_moves_only_the_length(dtype):
    """A start inside a block whose scale lies below what an append would write."""
    import torch
    H, d, block = 3, 64, 16
    c = filled(H, d, 64, block, dtype, [40] * H, 3)
    for s in (c.k_scale, c.v_scale):
        s[:, :3] = 2.0 ** -120
    before = [t.clone() for t in (c.K, c.V, c.k_scale, c.v_scale, c.mass)]
    empty = torch.empty(H, 0, d, device="cuda", dtype=_dt(dtype)[0])
    c.append(empty, empty, start=torch.tensor([37, 5, 64], dtype=torch.int32, device="cuda"))
    assert c.len.tolist() == [37, 5, 64] and c.status() == 0
    for t, b in zip((c.K, c.V, c.k_scale, c.v_scale, c.mass), before):
        assert torch.equal(t.view(torch.uint8), b.view(torch.uint8))
    c.append(empty, empty, start=torch.tensor([-1, 65, 7], dtype=torch.int32, device="cuda"))
    assert c.len.tolist() == [37, 5, 7] and c.status() == 5


# ------------------------------------------------------------------ small weights
@pytest.mark.parametrize("dtype,rows", KERNELS)
@pytest.mark.parametrize("apart", [12, 19, 20, 23, 27, 30, 33, 40])
def test_attend_channels_only_small_scales_fill(apart, dtype, rows):
    """Blocks of large V scale that are zero in half of the channels: the others come from tokens
    whose weight times scale is 2^-apart of the largest.  Full precision down to 2^-20, then
    what the smallest 16-bit weights hold (f32: all of it)."""
    import torch
    torch.manual_seed(apart)
    n, d, dt = 480, 64, _dt(dtype)[0]
    c = filled(1, d, 512, 16, dtype, [n], 5, max_queries=rows, spread=False)
    big = (torch.arange(n, device="cuda") // 16) % 3 == 0
    c.V[0, :n][big, d // 2:] = 0
    c.V[0, :n][~big, :d // 2] = 0
    c.v_scale[0, :n // 16] = torch.where(big[::16], 1.0, 2.0 ** -apart)
    c.K[0, :n] = 0                          # scores in one channel: 0 to 1/4, so that weights are not powers of two
    c.K[0, :n, 0] = (torch.rand(n, device="cuda") * 2).to(torch.float8_e4m3fn).view(torch.uint8)
    c.k_scale[0, :n // 16] = 1.0
    Q = torch.zeros(1, rows, d, dtype=dt, device="cuda")
    Q[0, :, 0] = torch.rand(rows, device="cuda").to(dt)
    O, lse = attend(c, Q)
    assert c.status() == 0
    ref = attend_one_head(c, 0, Q)
    K, V = head_values(c, 0)
    q = Q[0].double().cpu().numpy()
    w = np.exp(q @ K.T / np.sqrt(d))
    w /= w.sum(1, keepdims=True)
    scale = np.repeat(c.v_scale[0, :n // 16].double().cpu().numpy(), 16)
    codes = np.abs(host_codes(c.V[0, :n]))
    lost = 0.0
    if dtype == "bf16" and apart >= 20:
        lost = 2.0 ** -31 * (w * scale).max(1, keepdims=True) * codes.sum(0, keepdims=True)
    check_rows(O[0], lse[0], ref, None, dt, lost=lost)


# ------------------------------------------------------------------ queries
@pytest.mark.parametrize("dtype,rows", KERNELS)
@pytest.mark.parametrize("above", [4, 8, 9, 12, 14])
def test_queries_with_a_channel_far_above_the_rest(above, dtype, rows):
    """One query channel 2^above over the rest, K zero in it, heads of one token, whose lse is
    its score: elements down to 2^-9 of the largest enter a chunk whole, those of 16-row tiles
    down to 2^-14."""
    import torch
    torch.manual_seed(above)
    H, d, dt = 60, 128, _dt(dtype)[0]
    c = filled(H, d, 64, 64, dtype, [1] * H, 5, max_queries=rows)
    c.K[:, 0, 7] = 0
    Q = torch.rand(H, rows, d, device="cuda") + 1           # [1, 2): exponent 0 (2 after rounding up)
    Q *= torch.where(torch.rand(H, rows, d, device="cuda") < 0.5, -1.0, 1.0)
    Q[:, :, 7] = 2.0 ** above
    Q = Q.to(dt)
    O, lse = attend(c, Q)
    assert c.status() == 0
    chunk = dtype == "bf16" and rows >= 100
    for h in range(H):
        K, _ = head_values(c, h)
        more = 0.0
        if chunk and above > 9:
            more = 2.0 ** (above - 17) * np.abs(K[0]).sum() / np.sqrt(d)
        check_rows(O[h], lse[h], attend_one_head(c, h, Q), None, dt, dS_more=more)


# ------------------------------------------------------------------ K scales
@pytest.mark.parametrize("dtype,rows", KERNELS)
@pytest.mark.parametrize("exp", [-100, 112])
def test_mass_of_far_key_scales(exp, dtype, rows):
    """Keys and queries whose sizes make up for one another: scores and weights near 1."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    torch.manual_seed(rows)
    n, d, dt = 300, 128, _dt(dtype)[0]
    c = filled(1, d, 320, 64, dtype, [n], 2, max_queries=rows, spread=False)
    c.K[0, :n] = (448 - 128 * torch.rand(n, d, device="cuda")).to(torch.float8_e4m3fn).view(torch.uint8)
    c.k_scale[0, :5] = 2.0 ** exp
    Q = (2.0 ** -min(exp, 100) * (1 + torch.rand(1, rows, d, device="cuda"))).to(dt)
    scale = 2.0 ** (min(exp, 100) - exp - 17)
    O, lse = attend(c, Q, scale)
    check_attend(c, Q, O, lse, scale)
    c.accumulate(Q, lse, prev=torch.zeros_like(c.mass), scale=scale)
    assert c.status() == 0
    check_mass(c, Q, lse, 1.0, torch.zeros_like(c.mass), scale)


# ------------------------------------------------------------------ no tokens, one token
@pytest.mark.parametrize("dtype,rows", KERNELS)
@pytest.mark.parametrize("d", [64, 128])
def test_heads_that_hold_nothing_or_one_token(d, dtype, rows):
    """Every head empty: zeros, lse -inf, weights and a smaller cache left as they were; then one
    token each, in a graph that was captured over the empty cache."""
    import torch
    H, dt = 7, _dt(dtype)[0]
    torch.manual_seed(rows)
    c = poisoned(H, d, 64, 64, dtype, max_queries=rows)
    to = poisoned(H, d, 64, 64, dtype)
    Q = torch.randn(H, rows, d, device="cuda").to(dt)
    O, lse = torch.full_like(Q, 5.0), torch.full((H, rows), 5.0, device="cuda")

    def step():
        c.attend(Q, O, lse)
        c.accumulate(Q, lse)
        c.evict(to, 1)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for replay in (False, True):
        if replay:
            O.fill_(5.0)
            g.replay()
        assert bool((O == 0).all()) and bool(torch.isneginf(lse).all())
        assert bool(c.mass.isnan().all()) and to.len.tolist() == [0] * H
        for t in (to.K, to.V):
            assert bool((t == 0x7F).all())
    x = torch.randn(2, H, 1, d, device="cuda").to(dt)
    c.append(x[0], x[1])
    g.replay()
    assert c.status() == 0 and to.len.tolist() == [1] * H
    check_attend(c, Q, O, lse)
    # one token takes all of a row's weight: 1, but for its score's two roundings
    assert float((c.mass[:, 0] - rows).abs().max()) <= rows * 2.0 ** -10
    assert torch.equal(to.K[:, 0], c.K[:, 0]) and torch.equal(to.mass[:, 0], c.mass[:, 0])
