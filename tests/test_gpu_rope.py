"""GPU parity of kvb_rope with the fp64 oracle.

Tolerance: angles are formed and reduced in fp64, so cos and sin are within 2^-23 of
their values (an ulp and a half of 1, and the split remainder); x cos - y sin then is
off by at most (|x| + |y|) (2^-23 + 2^-24) for them, a product's rounding and the
sum's, together below (|x| + |y|) 2^-22; one rounding to the output type adds eps/2 of
the value."""
import numpy as np
import pytest

from oracle.rope import rope as oracle_rope

pytestmark = pytest.mark.gpu


def _check(got, x, pos, pairs, halves, inverse, bf16, base=10000.0):
    import torch
    ref = oracle_rope(x, pos, pairs, base, halves, inverse)
    d = x.shape[-1]
    i, j = (np.arange(d // 2), np.arange(d // 2) + d // 2) if halves else (np.arange(0, d, 2), np.arange(1, d, 2))
    size = np.zeros_like(ref)
    size[..., i] = size[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    half_step = torch.finfo(torch.bfloat16 if bf16 else torch.float32).eps / 2
    tol = (1 + half_step) * size * 2.0 ** -22 + half_step * np.abs(ref)
    assert np.all(np.abs(got - ref) <= tol), float((np.abs(got - ref) / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("heads,n,d,pairs", [(1, 1, 8, (1, 1, 1)), (12, 1, 128, (22, 21, 21)), (3, 7, 64, (12, 10, 10)),
                                             (5, 33, 72, (12, 12, 0)), (2, 130, 128, (64, 0, 0)),
                                             (40, 9, 256, (44, 42, 42)), (4, 65, 96, (0, 0, 0))])
def test_rope_matches_oracle(heads, n, d, pairs, halves, dtype):
    """Forwards and backwards, head-major and token-major rows on either side, rows
    padded to a longer stride, positions negative and far out."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    rng = np.random.default_rng(heads * 1000 + n + d)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    pos = rng.integers(-500, 100000, (n, 3)).astype(np.int32)
    pos[0] = [0, 2 ** 31 - 1, -2 ** 31] if n > 1 else [3, 5, 7]
    p = torch.from_numpy(pos).cuda()
    x = torch.randn(heads, n, d, device="cuda").to(dt)
    x64 = x.double().cpu().numpy()
    pair = kvb.KVB_ROPE_HALVES if halves else kvb.KVB_ROPE_INTERLEAVED
    for inverse in (False, True):
        for token_in, token_out, pad in ((False, False, 0), (True, False, 0), (False, True, 16)):
            src = torch.full((n, heads, d + pad) if token_in else (heads, n, d + pad), 7.0, device="cuda", dtype=dt)
            view = (src.transpose(0, 1) if token_in else src)[..., :d]
            view.copy_(x)
            dst = torch.full((n, heads, d + pad) if token_out else (heads, n, d + pad), 9.0, device="cuda", dtype=dt)
            out = (dst.transpose(0, 1) if token_out else dst)[..., :d]
            kvb.rope(view, p, out, pairs, pairing=pair, inverse=inverse)
            torch.cuda.synchronize()
            _check(out.double().cpu().numpy(), x64, pos, pairs, halves, inverse, dtype == "bf16")
            assert bool((dst[..., d:] == 9.0).all())          # the padding of the rows is left alone


def test_rope_in_place_and_gradient():
    """In place; and the inverse is the gradient: <rope(x), g> = <x, rope^-1(g)>, checked
    against a finite difference of the forward call and against the inner product."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    torch.manual_seed(0)
    H, n, d, pairs = 2, 50, 64, (12, 10, 10)
    pos = torch.randint(0, 3000, (n, 3), dtype=torch.int32, device="cuda")
    x, g, e = (torch.randn(H, n, d, device="cuda") for _ in range(3))
    y, dx, y1 = (torch.empty_like(x) for _ in range(3))
    kvb.rope(x, pos, y, pairs)
    kvb.rope(g, pos, dx, pairs, inverse=True)
    # both inner products: 6400 terms, each side's elements off by 2^-21 of its size at most
    size = float((y.double().abs() * g.double().abs()).sum())
    assert abs(float((y.double() * g.double()).sum() - (x.double() * dx.double()).sum())) <= 2.0 ** -19 * size
    kvb.rope(x + e, pos, y1, pairs)
    # linear: the difference over a whole step is the derivative; x + e rounds by 2^-24 of its size
    diff = float(((y1.double() - y.double()) * g.double()).sum())
    assert abs(diff - float((e.double() * dx.double()).sum())) <= 2.0 ** -18 * float(
        ((x.abs() + e.abs()) * (g.abs() + dx.abs())).double().sum())
    z = x.clone()
    kvb.rope(z, pos, z, pairs)
    assert torch.equal(z, y)


def test_rope_moves_a_key_to_frame_zero():
    """Rotating by the difference of positions takes a key from one position to another
    (a memory key's frame index set to 0)."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    torch.manual_seed(1)
    n, d, pairs = 64, 128, (22, 21, 21)
    pos = torch.randint(0, 50, (n, 3), dtype=torch.int32, device="cuda")
    x = torch.randn(3, n, d, device="cuda")
    a, b, c = (torch.empty_like(x) for _ in range(3))
    kvb.rope(x, pos, a, pairs)
    move = -pos
    move[:, 1:] = 0
    kvb.rope(a, move.contiguous(), b, pairs)
    at0 = pos.clone()
    at0[:, 0] = 0
    kvb.rope(x, at0, c, pairs)
    # three rotations, each within 2^-22 (|x| + |y|) and one fp32 rounding; pairs keep their norm
    assert float((b - c).abs().max()) <= 3 * (2 ** 0.5) * float(x.abs().max()) * (2.0 ** -21 + 2.0 ** -24) * 2


def test_rope_non_finite_values_stay_in_their_pair():
    import torch
    import kv_cache_compression_post_b200 as kvb
    x = torch.ones(1, 3, 32, device="cuda")
    x[0, 1, 4], x[0, 1, 31] = float("nan"), float("inf")
    pos = torch.full((3, 3), 2, dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)
    kvb.rope(x, pos, y, (4, 4, 4))          # pairs 12..15 (elements 24..31) are copied
    bad = ~torch.isfinite(y[0])
    want = torch.zeros_like(bad)
    want[1, 4] = want[1, 5] = want[1, 31] = True
    assert torch.equal(bad, want) and y[0, 1, 31] == float("inf") and y[0, 1, 30] == 1


def test_rope_far_strides_pass_32_bits():
    """Rows whose element offsets pass 2^31."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    step = 2 ** 30 + 64
    big = torch.empty(2 * step + 4096, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((3, 5, 64), (step, 64, 1))
    x.copy_(torch.randn(3, 5, 64, device="cuda"))
    pos = torch.randint(0, 100, (5, 3), dtype=torch.int32, device="cuda")
    y = torch.empty(3, 5, 64, dtype=torch.bfloat16, device="cuda")
    kvb.rope(x, pos, y, (12, 10, 10))
    _check(y.double().cpu().numpy(), x.double().cpu().numpy(), pos.cpu().numpy(), (12, 10, 10), False, False, True)
