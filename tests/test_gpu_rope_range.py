"""kvb_rope at the ends of its range: small and large bases, the furthest positions."""
import numpy as np
import pytest

from oracle.rope import rope as oracle_rope

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("base", [2.0 ** -21, 2.0 ** -10, 0.5, 1.0, 1e30])
@pytest.mark.parametrize("halves", [False, True])
def test_rope_stays_a_rotation(base, halves):
    """Any base and position keep every pair's norm, and give the oracle's values as far as fp64
    has the angle.  A frequency is 2^e with e = -log2(base) j / n, of three roundings (the
    logarithm's, the product's, the quotient's): 3 |e| 2^-53, which moves it by ln 2 times as
    much; the power and the product with the position add 2^-52 and 2^-53.  The oracle's exponent
    -j / n has one rounding, |e| 2^-53 again, and its power and product the same.  Together
    (4 ln 2 |e| + 6) 2^-53 of the angle."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    torch.manual_seed(3)
    H, d, pairs = 2, 64, (12, 10, 10)
    pos = torch.tensor([[0, 1, -1], [2 ** 31 - 1, -2 ** 31, 7], [-5, 12345, 2 ** 31 - 1], [1, 2 ** 20, -2 ** 31]],
                       dtype=torch.int32, device="cuda")
    x = torch.randn(H, 4, d, device="cuda")
    y = torch.empty_like(x)
    kvb.rope(x, pos, y, pairs, base=base, pairing=kvb.KVB_ROPE_HALVES if halves else kvb.KVB_ROPE_INTERLEAVED)
    i, j = (np.arange(32), np.arange(32) + 32) if halves else (np.arange(0, d, 2), np.arange(1, d, 2))
    a, b = x.double().cpu().numpy(), y.double().cpu().numpy()
    n0, n1 = np.hypot(a[..., i], a[..., j]), np.hypot(b[..., i], b[..., j])
    assert np.all(np.abs(n1 - n0) <= n0 * 2.0 ** -20)
    p = pos.cpu().numpy().astype(np.float64)
    angle = np.concatenate([np.abs(p[:, [k]]) * float(np.float32(base)) ** (-np.arange(m) / m)
                            for k, m in enumerate(pairs)], 1)
    e = np.concatenate([np.log2(base) * np.arange(m) / m for m in pairs])
    angle_off = angle * (4 * np.log(2) * np.abs(e) + 6) * 2.0 ** -53
    ref = oracle_rope(a, pos.cpu().numpy(), pairs, float(np.float32(base)), halves)
    tol = np.zeros_like(a)
    tol[..., i] = tol[..., j] = (np.abs(a[..., i]) + np.abs(a[..., j])) * (2.0 ** -21 + angle_off)
    assert np.all(np.abs(b - ref) <= tol)


@pytest.mark.parametrize("inverse", [False, True])
def test_rope_of_broadcast_rows(inverse):
    """Rows of X that lie on one another (a stride of 0): heads that share a key, tokens that share
    a row."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    torch.manual_seed(4)
    H, n, d, pairs = 5, 9, 64, (12, 10, 10)
    pos = torch.randint(-50, 3000, (n, 3), dtype=torch.int32, device="cuda")
    for x in (torch.randn(1, n, d, device="cuda").expand(H, n, d), torch.randn(H, 1, d, device="cuda").expand(H, n, d),
              torch.randn(1, 1, d, device="cuda").expand(H, n, d)):
        y, z = torch.empty(H, n, d, device="cuda"), torch.empty(H, n, d, device="cuda")
        kvb.rope(x, pos, y, pairs, inverse=inverse)
        kvb.rope(x.contiguous(), pos, z, pairs, inverse=inverse)
        assert torch.equal(y, z)
