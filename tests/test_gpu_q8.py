"""GPU parity of the 8-bit cache (kvb_q8_append / attend / mass / evict) with the fp64
oracle, on what the cache really holds.

Codes, scales, positions and kept weights are exact.  Attention and weights:

* A score is off by dS <= scale * sum_i |q_i k_i| * 2^-17: products are exact (the codes
  are, and Q's parts carry its 8 bits down to 2^-17 of a row's largest), 128 or fewer of
  them are summed in fp32 (each partial sum within 2^-23 of the absolute sum).  f32
  queries round each product and sum instead, the same bound.
* Every weight then is off by a factor exp(+-2 dS) (its own and the row's others'), the
  exponential adds 2^-18, and a weight held in fp16 2^-11: rel = 4 dS + 2^-11 + 2^-18.
* O = sum p v is off by rel * sum p |v|, and half a step of the output type.
* lse: dS, the exponentials' 2^-18, and fp32 sums and rounding 2^-17 (1 + |lse|).
* mass: a factor exp(dS) of each weight, 2^-18 for the exponential, the fp32 rounding of
  scores and lse 2^-23 (|s| + |lse|) each; prev's product and sum 2^-23.
"""
import numpy as np
import pytest

from oracle import q8cache as q8

pytestmark = pytest.mark.gpu

NAN_CODE = 0x7F


def _dt(dtype):
    import torch
    import kv_cache_compression_post_b200 as kvb
    return (torch.bfloat16, kvb.KVB_BF16) if dtype == "bf16" else (torch.float32, kvb.KVB_F32)


def host_codes(t):
    import torch
    return t.view(torch.float8_e4m3fn).double().cpu().numpy()


def poisoned(heads, d, cap, block, dtype, max_queries=1, with_mass=True):
    """A cache whose every byte behind the (zero) lengths is a NaN."""
    import kv_cache_compression_post_b200 as kvb
    c = kvb.Q8Cache(heads, d, cap, block, dtype=_dt(dtype)[1], max_queries=max_queries, with_mass=with_mass)
    c.K.fill_(NAN_CODE)
    c.V.fill_(NAN_CODE)
    for t in (c.k_scale, c.v_scale, c.mass):
        if t is not None:
            t.fill_(float("nan"))
    return c


def filled(heads, d, cap, block, dtype, lens, seed, max_queries=1, spread=True):
    """A poisoned cache with random codes and power-of-two scales below each length."""
    import torch
    c = poisoned(heads, d, cap, block, dtype, max_queries)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    for h, n in enumerate(lens):
        nb = -(-n // block)
        for code, scale in ((c.K, c.k_scale), (c.V, c.v_scale)):
            x = 64 * torch.randn(n, d, generator=g, device="cuda")
            code[h, :n] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            e = torch.randint(0, 4 if spread else 1, (nb,), generator=g, device="cuda")
            scale[h, :nb] = torch.exp2(-6.0 - e.float())
        c.mass[h, :n] = torch.rand(n, generator=g, device="cuda") ** 3
        c.len[h] = n
    return c


def head_values(c, h):
    n = int(c.len[h])
    K = q8.values(host_codes(c.K[h]), c.k_scale[h].double().cpu().numpy(), c.block, n)
    V = q8.values(host_codes(c.V[h]), c.v_scale[h].double().cpu().numpy(), c.block, n)
    return K, V


def attend(c, Q, scale=0.0, stream=None):
    import torch
    O = torch.full_like(Q, 123.0)
    lse = torch.full(Q.shape[:2], 123.0, device="cuda")
    c.attend(Q, O, lse, scale=scale, stream=stream)
    return O, lse


def check_attend(c, Q, O, lse, scale=0.0, rows=None):
    import torch
    half = torch.finfo(Q.dtype).eps / 2
    sc = scale or 1.0 / np.sqrt(Q.shape[2])
    for h in range(Q.shape[0]):
        K, V = head_values(c, h)
        pick = slice(None) if rows is None else rows
        q = Q[h, pick].double().cpu().numpy()
        ref, ref_lse, size = q8.attend(q, K, V, sc)
        got, got_lse = O[h, pick].double().cpu().numpy(), lse[h, pick].double().cpu().numpy()
        if len(K) == 0:
            assert np.all(got == 0) and np.all(np.isneginf(got_lse))
            continue
        dS = (np.abs(q) @ np.abs(K).T).max(1, keepdims=True) * sc * 2.0 ** -17
        rel = 4 * dS + 2.0 ** -11 + 2.0 ** -18
        tol = rel * size + half * (np.abs(ref) + rel * size)
        err = np.abs(got - ref)
        assert np.all(err <= tol), (h, float((err / tol).max()))
        el = np.abs(got_lse - ref_lse)
        tl = dS[:, 0] + 2.0 ** -18 + 2.0 ** -17 * (1 + np.abs(ref_lse))
        assert np.all(el <= tl), (h, float((el / tl).max()))


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,block", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 64), (128, 128)])
def test_append_matches_oracle(d, block, dtype):
    """Runs of every kind behind one another: single tokens, runs ending inside, at and
    behind a block's end, larger values later (older codes rounded anew), token-major and
    padded rows, a run of zeros, infinities and NaN."""
    import torch
    H, cap = 3, 1024
    torch.manual_seed(d + block)
    c = poisoned(H, d, cap, block, dtype)
    ref = [[(np.full((cap, d), np.nan), np.full(cap // block, np.nan)) for _ in range(2)] for _ in range(H)]
    at = 0
    for i, (n, size) in enumerate([(1, 1.0), (1, 3.0), (block - 2, 0.5), (block, 2.0), (2 * block + 1, 1.0), (1, 50.0),
                                   (3, 0.0), (block - 1, 1e-3), (5, 1e30), (block + 7, 1.0), (1, 1.0)]):
        K = (size * torch.randn(H, n, d, device="cuda")).to(_dt(dtype)[0])
        V = (size * torch.randn(n, H, d + 16, device="cuda")).to(_dt(dtype)[0])[..., :d].transpose(0, 1)
        if i == 3:
            K[1, 0, 3], K[2, 1, 5], K[2, 0, 0] = float("inf"), float("-inf"), float("nan")
        c.append(K, V)
        for h in range(H):
            for k, x in enumerate((K, V)):
                ref[h][k] = q8.append(*ref[h][k], block, at, x[h].double().cpu().numpy())
        at += n
        assert c.len.tolist() == [at] * H
    assert c.status() == 0
    for h in range(H):
        for k, (code, scale) in enumerate(((c.K, c.k_scale), (c.V, c.v_scale))):
            np.testing.assert_array_equal(host_codes(code[h]), ref[h][k][0])       # NaN behind the length too
            np.testing.assert_array_equal(scale[h].double().cpu().numpy(), ref[h][k][1])
        assert bool((c.mass[h, :at] == 0).all()) and bool(c.mass[h, at:].isnan().all())


def test_append_start_room_and_lengths():
    """A start of its own per head; heads without room are left as they were and say so."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    H, d, cap, block = 5, 64, 64, 16
    for n in (5, 40):                       # the one-launch and the two-launch form
        c = filled(H, d, cap, block, "f32", [20] * H, 3)
        before = [t.clone() for t in (c.K, c.V, c.k_scale, c.v_scale, c.mass)]
        K, V = torch.randn(2, H, n, d, device="cuda")
        start = torch.tensor([20, 7, cap - n, cap - n + 1, -1], dtype=torch.int32, device="cuda")
        c.append(K, V, start=start)
        assert c.len.tolist() == [20 + n, 7 + n, cap, 20, 20]
        assert c.status() == 5
        for h in (3, 4):
            for t, b in zip((c.K, c.V, c.k_scale, c.v_scale), before):
                assert torch.equal(t[h].view(torch.uint8), b[h].view(torch.uint8))
        for h, s in ((0, 20), (1, 7), (2, cap - n)):
            ref, rs = q8.append(host_codes(before[0][h]), before[2][h].double().cpu().numpy(), block, s,
                                K[h].double().cpu().numpy())
            np.testing.assert_array_equal(host_codes(c.K[h]), ref)
            np.testing.assert_array_equal(c.k_scale[h].double().cpu().numpy(), rs)
        empty = torch.empty(H, 0, d, device="cuda")
        c.append(empty, empty)              # nothing
        c.append(empty, empty, start=torch.full((H,), 9, dtype=torch.int32, device="cuda"))
        assert c.len.tolist() == [9] * H    # a length set back


@pytest.mark.parametrize("n", [3, 200])
def test_append_start_is_the_length(n):
    """start None, the length's own array and a copy of it are one call, room or no room, also
    behind one another."""
    import torch
    H, d, cap, block = 40, 64, 512, 16
    lens = [(37 * h) % 120 for h in range(H)]
    lens[3] = 480
    caches = [filled(H, d, cap, block, "bf16", lens, 9) for _ in range(3)]
    for _ in range(2):
        K, V = torch.randn(2, H, n, d, device="cuda").bfloat16()
        for c, start in zip(caches, (None, caches[1].len, caches[2].len.clone())):
            c.append(K, V, start=start)
    a = caches[0]
    room = [x + 2 * n <= cap for x in lens]
    assert a.len.tolist() == [x + 2 * n if r else x + n if x + n <= cap else x for x, r in zip(lens, room)]
    for b in caches[1:]:
        assert b.status() == a.status() == (0 if all(room) else 5)
        for x, y in zip((a.K, a.V, a.k_scale, a.v_scale, a.mass, a.len), (b.K, b.V, b.k_scale, b.v_scale, b.mass, b.len)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


# ------------------------------------------------------------------ attention
LENS = [0, 1, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 500]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 8, 9, 16, 17, 33, 49, 130])
@pytest.mark.parametrize("d,block", [(64, 16), (128, 64), (128, 128)])
def test_attend_ragged_lengths(d, block, rows, dtype):
    import torch
    torch.manual_seed(rows)
    c = filled(len(LENS), d, 512, block, dtype, LENS, rows, max_queries=rows)
    Q = (2 * torch.randn(len(LENS), rows, d, device="cuda")).to(_dt(dtype)[0])
    O, lse = attend(c, Q)
    assert c.status() == 0
    check_attend(c, Q, O, lse)
    O2, lse2 = attend(c, Q)                 # again: the same bits
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    c.attend(Q, O2.zero_(), None)           # without lse
    assert torch.equal(O, O2)


@pytest.mark.parametrize("rows", [1, 257, 300, 600])
@pytest.mark.parametrize("heads,lens", [(1, [5000]), (3, [4097, 129, 2000]), (40, None), (200, None)])
def test_attend_split_work(heads, lens, rows):
    """One long head cut over every CTA; lone row tiles; more heads than CTAs."""
    import torch
    if heads == 200 and rows > 300:
        rows = 40
    torch.manual_seed(heads + rows)
    lens = lens or [(37 * h) % 700 for h in range(heads)]
    c = filled(heads, 128, -(-max(lens) // 64) * 64, 64, "bf16", lens, heads, max_queries=rows)
    Q = torch.randn(heads, rows, 128, device="cuda").bfloat16()
    O, lse = attend(c, Q)
    assert c.status() == 0
    check_attend(c, Q, O, lse, rows=None if heads < 40 else np.array([0, rows // 2, rows - 1]))


@pytest.mark.parametrize("rows", [48, 49, 63, 80, 81])
@pytest.mark.parametrize("heads,cap", [(2, 65536), (3, 65536)])
def test_rows_between_the_kernels(heads, cap, rows):
    """Row counts on either side of the choice of kernel, for a small and a larger cache, with a
    workspace of exactly their size."""
    import torch
    c = filled(heads, 64, cap, 128, "bf16", [900, 0, 130][:heads], rows, max_queries=rows)
    Q = torch.randn(heads, rows, 64, device="cuda").bfloat16()
    c.mass.zero_()
    O, lse = attend(c, Q)
    c.accumulate(Q, lse)
    assert c.status() == 0
    check_attend(c, Q, O, lse)
    for h in range(heads):                  # every row's weights sum to 1
        n = int(c.len[h])
        assert abs(float(c.mass[h, :n].double().sum()) - (rows if n else 0)) <= rows * 2.0 ** -10
        assert bool((c.mass[h, n:] == 0).all())


@pytest.mark.parametrize("dtype,rows", [("bf16", 3), ("bf16", 140), ("f32", 3)])
def test_attend_sharp_and_scaled(dtype, rows):
    """Scores far apart (one token takes all), a late maximum, uneven scales of V by 2^40,
    scales that are no powers of two, and a scale argument."""
    import torch
    n, d, block = 400, 128, 16
    torch.manual_seed(5)
    c = filled(2, d, 400, block, dtype, [n, n - 3], 9, max_queries=rows)
    c.v_scale[0] = torch.exp2(-torch.randint(0, 40, (n // block,), device="cuda").float())
    c.k_scale[1] = 0.013 * (1 + torch.rand(n // block, device="cuda"))
    c.v_scale[1] = 0.3 * (1 + torch.rand(n // block, device="cuda"))
    Q = (6 * torch.randn(2, rows, d, device="cuda")).to(_dt(dtype)[0])
    K, _ = head_values(c, 0)
    Q[0, 0] = torch.from_numpy(3.0 * K[n - 2]).to(Q)        # its own token, at the end
    Q[1, 1] = 0                                              # uniform weights
    Q[1, 2] = Q[1, 2] * 1e-4
    for scale in (0.0, 0.4):
        O, lse = attend(c, Q, scale)
        check_attend(c, Q, O, lse, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [2, 200])
def test_attend_non_finite_queries_stay_in_their_row(rows, dtype):
    import torch
    torch.manual_seed(6)
    c = filled(2, 64, 256, 32, dtype, [200, 77], 4, max_queries=rows)
    Q = torch.randn(2, rows, 64, device="cuda").to(_dt(dtype)[0])
    clean, clean_lse = attend(c, Q)
    Q[0, 1, 5], Q[1, 0, 9] = float("nan"), float("inf")
    O, lse = attend(c, Q)
    for h, r in ((0, 1), (1, 0)):
        assert bool(O[h, r].isnan().all()) and bool(lse[h, r].isnan())
    keep = torch.ones(2, rows, dtype=torch.bool, device="cuda")
    keep[0, 1] = keep[1, 0] = False
    assert torch.equal(O[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])


@pytest.mark.parametrize("dtype,rows", [("bf16", 1), ("bf16", 20), ("bf16", 70), ("bf16", 100), ("f32", 3)])
def test_attend_scores_past_the_range_of_floats(rows, dtype):
    """The first 300 tokens' scores lie below -2^128 and count as -inf: they weigh nothing,
    and nothing else is touched."""
    import torch
    H, d, n, bad = 2, 128, 700, 300
    torch.manual_seed(rows)
    dt = _dt(dtype)[0]
    c = poisoned(H, d, 1024, 16, dtype, max_queries=rows)
    K, V = torch.randn(H, n, d, device="cuda"), torch.randn(H, n, d, device="cuda")
    K[:, :, 0] = 0.0
    K[:, :bad] = 0.0
    K[:, :bad, 0] = -2.0 ** 126
    c.append(K[:, :304].to(dt), V[:, :304].to(dt))
    c.append(K[:, 304:].to(dt), V[:, 304:].to(dt))
    Q = torch.randn(H, rows, d, device="cuda").to(dt)
    Q[:, :, 0] = 64.0
    O, lse = attend(c, Q)
    assert c.status() == 0
    # what is left: a cache without those tokens (300 = 18 blocks and 12 tokens; the four
    # that share a block with them lose their codes to its scale, and stay)
    one = poisoned(H, d, 1024, 16, dtype, max_queries=rows)
    for s, t in ((c.K, one.K), (c.V, one.V)):
        t[:, :n - 288] = s[:, 288:n]
    for s, t in ((c.k_scale, one.k_scale), (c.v_scale, one.v_scale)):
        t[:, :64 - 18] = s[:, 18:]
    one.len.fill_(n - 288)
    for h in range(H):
        Kh, Vh = head_values(one, h)
        assert np.all(Kh[:12, 0] == -2.0 ** 126) and np.all(Kh[12:16] == 0)
        q = Q[h].double().cpu().numpy()
        ref, ref_lse, size = q8.attend(q, Kh[12:], Vh[12:], 1.0 / np.sqrt(d))
        dS = (np.abs(q) @ np.abs(Kh[12:]).T).max(1, keepdims=True) / np.sqrt(d) * 2.0 ** -17
        rel = 4 * dS + 2.0 ** -11 + 2.0 ** -18
        half = torch.finfo(dt).eps / 2
        tol = rel * size + half * (np.abs(ref) + rel * size)
        assert np.all(np.abs(O[h].double().cpu().numpy() - ref) <= tol)
        tl = dS[:, 0] + 2.0 ** -18 + 2.0 ** -17 * (1 + np.abs(ref_lse))
        assert np.all(np.abs(lse[h].double().cpu().numpy() - ref_lse) <= tl)


def test_attend_lengths_out_of_range_and_poison():
    """A length past the capacity is the capacity, a negative one 0; nothing behind a
    length is read as a value (it is NaN here), rows behind stay as they were."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    for rows in (1, 150):
        c = filled(3, 128, 192, 64, "bf16", [192, 100, 50], 1, max_queries=rows)
        Q = torch.randn(3, rows, 128, device="cuda").bfloat16()
        want, _ = attend(c, Q)
        c.len[0] = 100000
        O, lse = attend(c, Q)
        assert torch.equal(O, want)
        c.len[1] = -7
        O, lse = attend(c, Q)
        assert bool((O[1] == 0).all()) and bool(torch.isneginf(lse[1]).all()) and torch.equal(O[2], want[2])


@pytest.mark.parametrize("rows", [1, 129])
def test_attend_offsets_past_32_bits(rows):
    """2^31 bytes of codes lie before the last head's tokens."""
    import torch
    H, d, cap = 9, 128, 1 << 21
    c = poisoned(H, d, cap, 128, "bf16", max_queries=rows, with_mass=False)
    n = 3000
    g = torch.Generator(device="cuda").manual_seed(0)
    for code, scale in ((c.K, c.k_scale), (c.V, c.v_scale)):
        code[H - 1, :n] = (64 * torch.randn(n, d, generator=g, device="cuda")).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[H - 1, :24] = 2.0 ** -6
    c.len[H - 1] = n
    Q = torch.randn(H, rows, d, device="cuda").bfloat16()
    O, lse = attend(c, Q)
    assert bool((O[:H - 1] == 0).all())
    small = filled(1, d, 3200, 128, "bf16", [0], 0, max_queries=rows)
    for a, b in ((small.K, c.K), (small.V, c.V), (small.k_scale, c.k_scale), (small.v_scale, c.v_scale)):
        a[0] = b[H - 1, :a.shape[1]]
    small.len[0] = n
    check_attend(small, Q[H - 1:], O[H - 1:], lse[H - 1:])


@pytest.mark.parametrize("name,H", [("wan480", 2), ("wan1080", 1)])
def test_attend_full_size_sampled_rows(name, H):
    """A chunk's queries over [sink | bank | window] of the 480P and 1080P workloads."""
    import torch
    import kvgen
    w = kvgen.WORKLOADS[name]
    n = w.F + w.capacity + w.chunk_tokens
    torch.manual_seed(7)
    c = filled(H, w.head_dim, -(-n // 64) * 64, 64, "bf16", [n - 13 * h for h in range(H)], 2,
               max_queries=w.chunk_tokens)
    Q = (1.5 * torch.randn(H, w.chunk_tokens, w.head_dim, device="cuda")).bfloat16()
    O, lse = attend(c, Q)
    assert c.status() == 0
    rows = np.sort(np.random.default_rng(0).choice(w.chunk_tokens, 24, replace=False))
    check_attend(c, Q, O, lse, rows=rows)


# ------------------------------------------------------------------ weights
def check_mass(c, Q, lse, decay, prev, scale=0.0):
    sc = scale or 1.0 / np.sqrt(Q.shape[2])
    for h in range(Q.shape[0]):
        n = int(c.len[h])
        K, _ = head_values(c, h)
        q, z = Q[h].double().cpu().numpy(), lse[h].double().cpu().numpy()
        got = c.mass[h].double().cpu().numpy()
        assert np.all(np.isnan(got[n:])), "weights behind the length changed"
        if n == 0:
            continue
        p = None if prev is None else prev[h, :n].double().cpu().numpy()
        ref = q8.mass(q, K, sc, z, decay, p)
        new = q8.mass(q, K, sc, z)
        fine = z[np.isfinite(z)]
        s = (np.abs(q) @ np.abs(K).T).max() * sc
        rel = 2 * s * 2.0 ** -17 + 2.0 ** -18 + 2.0 ** -22 * (s + (np.abs(fine).max() if len(fine) else 0))
        tol = rel * new + 2.0 ** -20 * new + 2.0 ** -22 * np.abs(ref - new) + len(q) * 2.0 ** -126
        err = np.abs(got[:n] - ref)
        assert np.all(err <= tol), (h, float((err / tol).max()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 16, 17, 130, 300])
@pytest.mark.parametrize("d,block", [(64, 16), (128, 64)])
def test_mass_matches_oracle(d, block, rows, dtype):
    import torch
    torch.manual_seed(rows + d)
    c = filled(len(LENS), d, 512, block, dtype, LENS, rows, max_queries=rows)
    Q = (2 * torch.randn(len(LENS), rows, d, device="cuda")).to(_dt(dtype)[0])
    _, lse = attend(c, Q)
    lse[3, rows // 2] = float("-inf")                      # a row that saw nothing weighs nothing
    prev = c.mass.clone()
    c.accumulate(Q, lse, decay=0.5)                        # onto its own weights
    assert c.status() == 0
    check_mass(c, Q, lse, 0.5, prev)
    first = c.mass.clone()
    c.mass.copy_(prev)
    c.accumulate(Q, lse, decay=0.5, prev=prev)             # onto others: the same bits
    assert torch.equal(c.mass.view(torch.int32), first.view(torch.int32))
    held = torch.arange(512, device="cuda") < c.len[:, None]
    import kv_cache_compression_post_b200 as kvb
    c.mass.fill_(float("nan"))
    kvb.kvb_q8_mass(c.c, Q, rows, c.dtype, 0.0, lse, 0.5, None, c.ws, c.nbytes)   # onto none
    total = torch.where(held, c.mass, torch.zeros_like(c.mass)).double().sum(1).cpu().numpy()
    want = np.array([0.0 if n == 0 else rows - (h == 3) for h, n in enumerate(LENS)])
    # each row's weights sum to 1, but for the errors of a score (see above) on either side
    np.testing.assert_allclose(total, want, rtol=2e-3)


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("rows,dtype", [(1, "bf16"), (20, "bf16"), (300, "bf16"), (1, "f32"), (5, "f32")])
def test_mass_of_rows_that_saw_nothing(rows, dtype):
    """Rows of lse -inf weigh nothing: what was there before stays to the bit."""
    import torch
    c = filled(2, 128, 512, 64, dtype, [500, 0], rows, max_queries=rows)
    prev = torch.rand(2, 512, device="cuda") * 2.0 ** -110
    Q = torch.randn(2, rows, 128, device="cuda").to(_dt(dtype)[0])
    c.accumulate(Q, torch.full((2, rows), float("-inf"), device="cuda"), prev=prev)
    assert torch.equal(c.mass[0, :500], prev[0, :500])


@pytest.mark.parametrize("d,block", [(64, 16), (128, 64), (128, 128)])
@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (100, 0, 0), (100, 7, 30), (100, 40, 60), (300, 1, 299),
                                                (333, 16, 64), (2000, 5, 5)])
def test_evict_matches_oracle(d, block, budget, sink, recent):
    import torch
    import kv_cache_compression_post_b200 as kvb
    lens = [0, 1, 99, 100, 101, 333, 334, 1500, 2000]
    H, cap = len(lens), 2048
    c = filled(H, d, cap, block, "bf16", lens, budget)
    c.mass[5, :300] = 0.25                                  # ties across the cut
    c.mass[6, :334:3] = 0.0
    c.mass[6, 1:334:3] = -0.0
    c.mass[7, 100:900] = float("nan")
    c.mass[7, 901], c.mass[8, 3], c.mass[8, 4] = float("inf"), float("-inf"), -1.0
    c.mass[8, 1000:] = c.mass[8, 1000]
    to = poisoned(H, d, -(-budget // block) * block, block, "bf16")
    kept = torch.full((H, budget), -5, dtype=torch.int32, device="cuda")
    before = [t.clone() for t in (c.K, c.V, c.k_scale, c.v_scale, c.mass, c.len)]
    c.evict(to, budget, sink=sink, recent=recent, kept=kept)
    for t, b in zip((c.K, c.V, c.k_scale, c.v_scale, c.mass, c.len), before):
        assert torch.equal(t.view(torch.uint8), b.view(torch.uint8)), "the source changed"
    w = c.mass.double().cpu().numpy()
    for h, n in enumerate(lens):
        want = q8.keep(w[h], n, budget, sink, recent)
        m = len(want)
        assert int(to.len[h]) == m == min(n, budget)
        np.testing.assert_array_equal(kept[h, :m].cpu().numpy(), want)
        assert bool((kept[h, m:] == -5).all())
        np.testing.assert_array_equal(to.mass[h, :m].double().cpu().numpy(), w[h][want])
        assert bool(to.mass[h, m:].isnan().all())
        for a, s, b, z in ((c.K, c.k_scale, to.K, to.k_scale), (c.V, c.v_scale, to.V, to.v_scale)):
            got = host_codes(b[h])
            assert np.all(np.isnan(got[m:]))
            if m == 0:
                continue
            codes, scales = q8.gather(host_codes(a[h]), s[h].double().cpu().numpy(), block, want)
            np.testing.assert_array_equal(got[:m], codes)
            np.testing.assert_array_equal(z[h, :len(scales)].double().cpu().numpy(), scales)
    # without the list, and without weights of its own
    two = kvb.Q8Cache(H, d, to.capacity, block)
    c.evict(two, budget, sink=sink, recent=recent)
    assert torch.equal(two.len, to.len)
    for h in range(H):
        m = int(to.len[h])
        assert torch.equal(two.K[h, :m], to.K[h, :m]) and torch.equal(two.V[h, :m], to.V[h, :m])


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype,d,halves", [("bf16", 128, False), ("f32", 64, True)])
def test_rotate_append_attend_weigh_evict(dtype, d, halves):
    """Two chunks, then single tokens, as a streaming generator would: rotate, append,
    attend, accumulate the weights, cut to a budget, go on in the cut cache."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    from oracle.rope import rope as oracle_rope
    torch.manual_seed(11)
    H, block, chunk, budget, sink, recent = 3, 32, 170, 260, 17, 40
    dt, code = _dt(dtype)
    pairs = (d // 2 - 2 * (d // 6), d // 6, d // 6)
    a = kvb.Q8Cache(H, d, 512, block, dtype=code, max_queries=chunk, with_mass=True)
    b = kvb.Q8Cache(H, d, 512, block, dtype=code, max_queries=chunk, with_mass=True)
    ref = [[np.zeros((512, d)), np.zeros(512 // block)] for _ in range(2 * H)]
    at, length = 0, 0
    for n in (chunk, chunk, 1, 1, 5):
        pos = torch.stack([torch.arange(at, at + n) // 17, torch.arange(n) // 5, torch.arange(n) % 5], 1).int().cuda()
        x = torch.randn(3, n, H, d, device="cuda").to(dt)
        q, k, out = (torch.empty(H, n, d, device="cuda", dtype=dt) for _ in range(3))
        lse = torch.empty(H, n, device="cuda")
        pairing = kvb.KVB_ROPE_HALVES if halves else kvb.KVB_ROPE_INTERLEAVED
        kvb.rope(x[0].transpose(0, 1), pos, q, pairs, pairing=pairing)
        kvb.rope(x[1].transpose(0, 1), pos, k, pairs, pairing=pairing)
        want = oracle_rope(x[1].transpose(0, 1).double().cpu().numpy(), pos.cpu().numpy(), pairs, halves=halves)
        assert np.abs(k.double().cpu().numpy() - want).max() <= np.abs(want).max() * torch.finfo(dt).eps
        v = x[2].transpose(0, 1)
        prev = a.mass.clone()
        a.append(k, v)
        a.attend(q, out, lse)
        a.accumulate(q, lse, decay=0.75)
        for h in range(H):
            for i, y in enumerate((k, v)):
                r = ref[2 * h + i]
                r[0], r[1] = q8.append(r[0], r[1], block, length, y[h].double().cpu().numpy())
                got = host_codes((a.K, a.V)[i][h])
                np.testing.assert_array_equal(got[:length + n], r[0][:length + n])
        length += n
        at += n
        assert a.len.tolist() == [length] * H and a.status() == 0
        check_attend(a, q, out, lse)
        prev[:, length - n:length] = 0
        for h in range(H):
            K, _ = head_values(a, h)
            w = q8.mass(q[h].double().cpu().numpy(), K, d ** -0.5, lse[h].double().cpu().numpy(), 0.75,
                        prev[h, :length].double().cpu().numpy())
            # scores here stay below 40: 2^-17 * 40 and the exponential, twice over
            np.testing.assert_allclose(a.mass[h, :length].double().cpu().numpy(), w, rtol=1e-3, atol=1e-12)
        if length > budget:
            kept = torch.empty(H, budget, dtype=torch.int32, device="cuda")
            a.evict(b, budget, sink=sink, recent=recent, kept=kept)
            for h in range(H):
                idx = q8.keep(a.mass[h].double().cpu().numpy(), length, budget, sink, recent)
                np.testing.assert_array_equal(kept[h].cpu().numpy(), idx)
                for i in range(2):
                    r = ref[2 * h + i]
                    codes, scales = q8.gather(r[0], r[1], block, idx)
                    r[0], r[1] = np.zeros((512, d)), np.zeros(512 // block)
                    r[0][:budget], r[1][:len(scales)] = codes, scales
            a, b, length = b, a, budget


def test_captured_decode_loop():
    """A captured (append, attend, accumulate) step follows the device-side lengths when
    replayed, and equals the same steps run one by one."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    torch.manual_seed(12)
    H, d, block, n0, steps = 4, 128, 64, 100, 70
    caches = [filled(H, d, 256, block, "bf16", [n0] * H, 5) for _ in range(2)]
    for c in caches:
        c.mass.zero_()
    xs = torch.randn(steps, 3, H, 1, d, device="cuda").bfloat16()
    x = torch.empty_like(xs[0])
    O = [torch.empty(H, 1, d, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    lse = [torch.empty(H, 1, device="cuda") for _ in range(2)]

    def step(i):
        c = caches[i]
        c.append(x[0], x[1])
        c.attend(x[2], O[i], lse[i])
        c.accumulate(x[2], lse[i])

    step(0)
    torch.cuda.synchronize()
    warm = [t.clone() for t in (caches[1].K, caches[1].V, caches[1].k_scale, caches[1].v_scale, caches[1].mass)]
    caches[0] = filled(H, d, 256, block, "bf16", [n0] * H, 5)
    caches[0].mass.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(1)
    assert caches[1].len.tolist() == [n0] * H               # capturing ran nothing
    for t, w in zip((caches[1].K, caches[1].V, caches[1].k_scale, caches[1].v_scale, caches[1].mass), warm):
        assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))
    for s in range(steps):
        x.copy_(xs[s])
        step(0)
        g.replay()
        assert torch.equal(O[0], O[1]) and torch.equal(lse[0], lse[1])
    assert caches[1].len.tolist() == [n0 + steps] * H
    for a, b in ((caches[0].K, caches[1].K), (caches[0].k_scale, caches[1].k_scale), (caches[0].mass, caches[1].mass)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    check_attend(caches[1], x[2], O[1], lse[1])


def test_two_streams_and_two_caches_at_once():
    """Calls on different caches overlap on two streams and give what they give alone."""
    import torch
    torch.manual_seed(13)
    H, d, rows = 6, 128, 300
    caches = [filled(H, d, 2048, 64, "bf16", [2000 - 100 * h for h in range(H)], s, max_queries=rows) for s in (1, 2)]
    Q = [torch.randn(H, rows, d, device="cuda").bfloat16() for _ in range(2)]
    want = []
    for c, q in zip(caches, Q):
        O, lse = attend(c, q)
        prev = c.mass.clone()
        c.accumulate(q, lse, prev=prev)
        want.append((O, lse, c.mass.clone(), prev))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(2):
        O, lse = torch.empty_like(Q[i]), torch.empty(H, rows, device="cuda")
        got.append((O, lse))
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                caches[i].attend(Q[i], *got[i])
                caches[i].accumulate(Q[i], got[i][1], prev=want[i][3])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])
        assert torch.equal(caches[i].mass.view(torch.int32), want[i][2].view(torch.int32))
        assert caches[i].status() == 0


# ------------------------------------------------------------------ edges of the calls
def test_captured_chunk_step_and_eviction():
    """A captured step of a chunk (append, attend, accumulate, evict into a second cache) and
    its replays, in a workspace that a second captured graph uses in turn."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    torch.manual_seed(21)
    H, d, block, n, rows = 3, 128, 64, 300, 200
    a = kvb.Q8Cache(H, d, 1024, block, max_queries=rows, with_mass=True)
    b = kvb.Q8Cache(H, d, 512, block, max_queries=rows, with_mass=True)
    b.ws, b._buf = a.ws, a._buf                       # one workspace, used one call after another
    x = torch.randn(3, H, n, d, device="cuda").bfloat16()
    Q = torch.randn(H, rows, d, device="cuda").bfloat16()
    one = torch.randn(H, 2, d, device="cuda").bfloat16()
    O, lse = torch.empty_like(Q), torch.empty(H, rows, device="cuda")
    O2, lse2 = torch.empty_like(one), torch.empty(H, 2, device="cuda")

    def chunk():
        a.append(x[0], x[1])
        a.attend(Q, O, lse)
        a.accumulate(Q, lse)
        a.evict(b, 256, sink=5, recent=20)

    def token():
        b.attend(one, O2, lse2)
        b.accumulate(one, lse2, decay=0.5)

    chunk(), token()
    torch.cuda.synchronize()
    want = [t.clone() for t in (O, lse, a.mass, b.K, b.V, b.mass, O2, lse2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, f in zip(graphs, (chunk, token)):
        with torch.cuda.graph(g):
            f()
    for _ in range(3):
        a.len.zero_()
        a.mass.zero_()
        b.mass.zero_()
        for g in graphs:
            g.replay()
        for got, w in zip((O, lse, a.mass, b.K, b.V, b.mass, O2, lse2), want):
            if got is b.K or got is b.V:
                got, w = got[:, :256], w[:, :256]
            assert torch.equal(got, w)
    assert a.status() == 0 and b.status() == 0
    check_attend(a, Q, O, lse)
    check_attend(b, one, O2, lse2)


@pytest.mark.parametrize("rows", [1, 12, 40, 300])
def test_workspace_needs_no_initialisation(rows):
    """Whatever the workspace held, also between calls of another kind, changes nothing."""
    import torch
    torch.manual_seed(rows)
    c = filled(2, 128, 8192, 64, "bf16", [8000, 5000], 3, max_queries=300)
    Q = torch.randn(2, rows, 128, device="cuda").bfloat16()
    O, lse = attend(c, Q)
    prev = c.mass.clone()
    c.accumulate(Q, lse, prev=prev)
    mass = c.mass.clone()
    for fill in (0, 255, None):
        if fill is None:
            c._buf.random_(0, 256)
        else:
            c._buf.fill_(fill)
        O2, lse2 = attend(c, Q)
        assert torch.equal(O, O2) and torch.equal(lse, lse2)
        c.accumulate(Q, lse, prev=prev)
        assert torch.equal(c.mass.view(torch.int32), mass.view(torch.int32))
    check_attend(c, Q, O, lse, rows=np.array([0, rows - 1]))


@pytest.mark.parametrize("low", [1e-30, 0.999, -1.0, float("nan")])
@pytest.mark.parametrize("more", [-1, 0, 1])
def test_evict_where_a_digit_decides(low, more):
    """Two weights, and a budget of as many as have the larger, one less and one more: all keys
    of a digit stay, at the first or a later digit, or all but one."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    n, sink, recent = 5000, 3, 5
    c = filled(2, 64, 5008, 16, "bf16", [n, n - 1], 1)
    mass = torch.full((n,), low, device="cuda")
    mass[sink + 1:n - recent - 1:3] = 1.0
    c.mass[:, :n] = mass
    budget = int((mass == 1.0).sum()) + sink + recent + more
    to = kvb.Q8Cache(2, 64, -(-budget // 16) * 16, 16)
    kept = torch.empty(2, budget, dtype=torch.int32, device="cuda")
    c.evict(to, budget, sink=sink, recent=recent, kept=kept)
    for h, m in enumerate((n, n - 1)):
        want = q8.keep(c.mass[h].double().cpu().numpy(), m, budget, sink, recent)
        np.testing.assert_array_equal(kept[h].cpu().numpy(), want)


def test_evict_more_tokens_than_shared_memory_holds():
    """200001 tokens of one head (a cluster keeps the keys of 131072 between its passes), and
    a budget of none but ties."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    n, budget = 200001, 70000
    c = kvb.Q8Cache(1, 64, 200064, 64, with_mass=True)
    c.K.random_(0, 100)
    c.V.random_(0, 100)
    c.k_scale.fill_(0.5)
    c.v_scale.fill_(0.25)
    c.len.fill_(n)
    to = kvb.Q8Cache(1, 64, 70016, 64)
    kept = torch.empty(1, budget, dtype=torch.int32, device="cuda")
    for mass in (torch.rand(200064, device="cuda"), torch.full((200064,), 3.0, device="cuda")):
        c.mass[0] = mass
        c.evict(to, budget, sink=11, recent=501, kept=kept)
        w = mass[:n].clone()
        w[:11] = w[n - 501:] = float("inf")
        want = w.sort(descending=True, stable=True)[1][:budget].sort()[0]
        assert torch.equal(kept[0].long(), want) and to.len.item() == budget
        assert torch.equal(to.K[0, :budget], c.K[0, want]) and torch.equal(to.V[0, :budget], c.V[0, want])


@pytest.mark.parametrize("listed", [False, True])
def test_evict_into_a_larger_cache(listed):
    """A budget above the source's capacity keeps all, and nothing behind the workspace or
    the list is written."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    H, cap, budget = 64, 16, 65536
    lens = [(7 * h) % (cap + 1) for h in range(H)]
    c = filled(H, 64, cap, 16, "bf16", lens, 5)
    to = kvb.Q8Cache(H, 64, budget, 16, with_mass=True)
    kept = torch.full((H, budget), -5, dtype=torch.int32, device="cuda") if listed else None
    buf = torch.full((c.nbytes + (32 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    ws = (buf.data_ptr() + 255) & ~255
    end = ws - buf.data_ptr() + c.nbytes
    kvb.kvb_q8_evict(c.c, to.c, budget, 3, budget - 3, kept, ws, c.nbytes)
    assert bool((buf[end:] == 0xA5).all())
    assert to.len.tolist() == lens
    for h, n in enumerate(lens):
        assert torch.equal(to.K[h, :n], c.K[h, :n]) and torch.equal(to.V[h, :n], c.V[h, :n])
        assert torch.equal(to.mass[h, :n], c.mass[h, :n])
        if listed:
            assert kept[h, :n].tolist() == list(range(n)) and bool((kept[h, n:] == -5).all())


def test_attend_work_past_32_bits():
    """A split whose costs times the CTAs pass 2^32: 80 heads, 24000 queries, 65536 tokens."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    H, rows, n = 80, 24000, 65536
    c = kvb.Q8Cache(H, 64, n, 128, max_queries=rows)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(n, 64, generator=g, device="cuda")
    c.K[:] = (64 * x).to(torch.float8_e4m3fn).view(torch.uint8)
    c.V[:] = (64 * x.flip(0)).to(torch.float8_e4m3fn).view(torch.uint8)
    c.k_scale.fill_(2.0 ** -6)
    c.v_scale.fill_(2.0 ** -6)
    c.len.fill_(n)
    Q = torch.randn(1, rows, 64, generator=g, device="cuda").bfloat16().expand(H, -1, -1).contiguous()
    O, lse = attend(c, Q)
    assert c.status() == 0
    assert torch.equal(lse.isfinite().sum(), torch.tensor(H * rows, device="cuda"))
    one = kvb.Q8Cache(1, 64, n, 128, max_queries=rows)
    for s, t in ((c.K, one.K), (c.V, one.V), (c.k_scale, one.k_scale), (c.v_scale, one.v_scale), (c.len, one.len)):
        t.copy_(s[:1])
    for h in (0, 41, H - 1):
        check_attend(one, Q[h:h + 1], O[h:h + 1], lse[h:h + 1], rows=np.array([0, 11111, rows - 1]))
    # the same inputs in every head: the same outputs, but for where a unit was cut
    assert float((O.float() - O[:1].float()).abs().max()) <= 2.0 ** -7 * float(O[0].float().abs().max())


def test_binding_refuses_wrong_tensors_and_devices():
    import torch
    import kv_cache_compression_post_b200 as kvb
    H, d = 2, 64
    c = kvb.Q8Cache(H, d, 128, 64, max_queries=4)
    Q = torch.zeros(H, 4, d, device="cuda", dtype=torch.bfloat16)
    O, lse = torch.empty_like(Q), torch.empty(H, 4, device="cuda")
    bad = [lambda: c.attend(Q.float(), O, lse), lambda: c.attend(Q, O.float(), lse), lambda: c.attend(Q, O[:, :3], lse),
           lambda: c.attend(Q.cpu(), O, lse), lambda: c.attend(Q, O, lse.double()), lambda: c.attend(Q, O, lse[:1]),
           lambda: c.attend(Q[:1], O[:1], lse[:1]), lambda: c.attend(Q[..., ::2], O[..., ::2], lse),
           lambda: c.attend(Q.transpose(0, 1).contiguous().transpose(0, 1), O, lse), lambda: c.attend(Q[0], O[0], lse[0]),
           lambda: c.attend(Q[:, :0], O[:, :0], lse[:, :0]),
           lambda: c.append(Q, Q[:, :2]), lambda: c.append(Q, Q.float()), lambda: c.append(Q[..., ::2], Q[..., ::2]),
           lambda: c.append(Q, Q, start=torch.zeros(H, device="cuda")), lambda: c.append(Q.cpu(), Q.cpu()),
           lambda: c.accumulate(Q, lse), lambda: c.evict(kvb.Q8Cache(H, d, 64, 64), 10),
           lambda: kvb.Q8Cache(H, d, 100, 64), lambda: kvb.Q8Cache(H, 96, 128, 64), lambda: kvb.Q8Cache(H, d, 128, 64, K=O),
           lambda: kvb.rope(Q, torch.zeros(4, 3, device="cuda"), O, (1, 1, 1)),
           lambda: kvb.rope(Q, torch.zeros(4, 3, dtype=torch.int32), O, (1, 1, 1)),
           lambda: kvb.rope(Q, torch.zeros(4, 3, dtype=torch.int32, device="cuda"), O, (30, 2, 1)),
           lambda: kvb.rope(Q, torch.zeros(4, 3, dtype=torch.int32, device="cuda"), O, (1, 1))]
    for i, f in enumerate(bad):
        with pytest.raises(kvb.KvbError) as e:
            f()
        assert e.value.status in (1, 7), i
    big = torch.zeros(H, 300, d, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(kvb.KvbError) as e:               # more queries than the workspace is for
        c.attend(big, big.clone())
    assert e.value.status == 2
    c.device = 1                                         # a cache of another device than the current one
    with pytest.raises(kvb.KvbError) as e:
        c.attend(Q, O, lse)
    assert e.value.status == 1
