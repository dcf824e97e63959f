"""Pins of oracle/rope.py and oracle/q8cache.py (CPU)."""
import numpy as np
import pytest

import kvgen
from oracle import q8cache as q8
from oracle.attention import attention
from oracle.fp8 import e4m3
from oracle.rope import rope


def test_rope_is_the_generators_rotation():
    """The backbone's 3D rotation, which kvgen applies to what the workloads' caches hold."""
    d, rng = 128, np.random.default_rng(0)
    pos = np.stack([rng.integers(0, 200, 40), rng.integers(0, 30, 40), rng.integers(0, 52, 40)], 1)
    x = rng.standard_normal((3, 40, d)).astype(np.float32)
    want = kvgen.apply_rope(x, kvgen.rope_angles(d, pos[:, 0], pos[:, 1], pos[:, 2]))
    np.testing.assert_allclose(rope(x, pos, kvgen.rope_pairs(d)), want, atol=2e-6)


@pytest.mark.parametrize("halves", [False, True])
def test_rope_inverse_norms_and_copied_pairs(halves):
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((2, 9, 48)), rng.integers(-50, 5000, (9, 3))
    y = rope(x, pos, (7, 6, 5), halves=halves)
    np.testing.assert_allclose(rope(y, pos, (7, 6, 5), halves=halves, inverse=True), x, atol=1e-12)
    np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-12)
    kept = np.r_[18:24, 42:48] if halves else np.r_[36:48]
    assert np.array_equal(y[..., kept], x[..., kept])
    # scores depend on differences of positions only: q.k after a common shift
    s = rope(x, pos + 11, (7, 6, 5), halves=halves)
    np.testing.assert_allclose(y[0] @ y[1].T, s[0] @ s[1].T, atol=1e-9)


def test_block_scale_is_the_smallest_power_of_two():
    for m, e in [(448.0, 0), (448.5, 1), (1.0, -8), (1.75, -8), (1.7500001, -7), (0.0, -100), (3e38, 119)]:
        assert q8.block_scale([m, -m / 2]) == 2.0 ** e, m
    assert q8.block_scale([np.inf, 1.0, np.nan]) == 2.0 ** -8


def test_append_keeps_the_larger_scale_and_rounds_older_codes_anew():
    rng = np.random.default_rng(2)
    codes, scales = np.zeros((64, 8)), np.ones(4)
    a, b = rng.standard_normal((20, 8)), 40 * rng.standard_normal((5, 8))
    codes, scales = q8.append(codes, scales, 16, 0, a)
    first = codes.copy(), scales.copy()
    codes, scales = q8.append(codes, scales, 16, 20, b)
    assert np.array_equal(codes[:16], first[0][:16]) and scales[0] == first[1][0]
    assert scales[1] > first[1][1]
    got = q8.values(codes, scales, 16, 25)
    np.testing.assert_allclose(got[20:], b, rtol=2.0 ** -4, atol=scales[1] * 2.0 ** -10)
    assert np.array_equal(got[16:20], scales[1] * e4m3(first[0][16:20] * first[1][1] / scales[1]))


def test_attention_weights_and_eviction():
    rng = np.random.default_rng(3)
    Q, K, V = rng.standard_normal((5, 8)), rng.standard_normal((30, 8)), rng.standard_normal((30, 8))
    O, lse, _ = q8.attend(Q, K, V, 0.3)
    O2, lse2 = attention(Q, K, V, 0.3)
    np.testing.assert_allclose(O, O2, atol=1e-12)
    np.testing.assert_allclose(lse, lse2, atol=1e-12)
    w = q8.mass(Q, K, 0.3, lse)
    assert abs(w.sum() - 5) < 1e-12          # each row's weights sum to 1
    kept = q8.keep(w, 30, 12, 2, 3)
    assert len(kept) == 12 and set(kept) >= {0, 1, 27, 28, 29}
    mid = [i for i in kept if 2 <= i < 27]
    out = [i for i in range(2, 27) if i not in mid]
    assert min(w[mid]) >= max(w[out])
    assert np.array_equal(q8.keep(np.ones(10), 10, 4, 0, 1), [0, 1, 2, 9])
    assert np.array_equal(q8.keep(np.array([np.nan, -np.inf, 0.0, -0.0]), 4, 3, 0, 0), [1, 2, 3])
