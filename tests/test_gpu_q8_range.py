"""The 8-bit cache's calls at the ends of their ranges: scores, scales, queries and log sums
far from 1, weights too small for the 16 bits they are held in.

Tolerances are those of test_gpu_q8.py (a score is off by dS, a weight by a factor
1 + rel), widened where a test says so.
"""
import numpy as np
import pytest

from oracle import q8cache as q8
from tests.test_gpu_q8 import _dt, attend, check_mass, filled, head_values

pytestmark = pytest.mark.gpu

# every kernel: few rows, 16-row tiles (one and several), chunks (a lone tile, a pair), f32
KERNELS = [("bf16", 1), ("bf16", 8), ("bf16", 12), ("bf16", 40), ("bf16", 100), ("bf16", 300), ("f32", 1), ("f32", 5)]


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


# ------------------------------------------------------------------ scores
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
