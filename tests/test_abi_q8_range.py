"""Host-side refusals at the ends of the calls' ranges (no GPU: every check returns before
anything is launched)."""
import ctypes

P = ctypes.c_void_p(0x10000)       # never dereferenced


def _cache():
    import kv_cache_compression_post_b200 as kvb
    return kvb.kvb_q8_cache(heads=1, head_dim=64, capacity=256, block=64, K=0x1000, V=0x2000, k_scale=0x3000,
                            v_scale=0x4000, len=0x5000, mass=0x6000, status=0x7000)


def test_row_counts_past_the_range():
    """The workspace grows with the rows up to 2^30 of them; more are refused everywhere."""
    import kv_cache_compression_post_b200 as kvb
    c = _cache()
    for dtype in (kvb.KVB_BF16, kvb.KVB_F32):
        sizes = [kvb.kvb_q8_workspace_size(c, n, dtype) for n in (1, 1 << 20, 1 << 29, 1 << 30)]
        assert 0 < sizes[0] and sizes == sorted(sizes)
        for n in ((1 << 30) + 1, (1 << 31) - 256, (1 << 31) - 1):
            assert kvb.kvb_q8_workspace_size(c, n, dtype) == 0, n
            assert kvb.lib.kvb_q8_attend(ctypes.byref(c), P, n, dtype, 0.0, P, P, P, 1 << 60, None) == 1
            assert kvb.lib.kvb_q8_mass(ctypes.byref(c), P, n, dtype, 0.0, P, 1.0, None, P, 1 << 60, None) == 1


def test_rope_bases_whose_angles_pass_whole_turns():
    """A base below 2^-21 turns far positions by more than 2^52 rad, of which fp64 has no fraction."""
    import kv_cache_compression_post_b200 as kvb
    pairs = (ctypes.c_int32 * 3)(12, 10, 10)

    def f(base, n):
        return kvb.lib.kvb_rope(P, P, 2, n, 64, 0, pairs, base, 0, 0, 320, 64, P, 320, 64, None)

    for base in (1e-45, 1e-30, 1e-10, 2.0 ** -21 * (1 - 2.0 ** -23)):
        assert f(base, 5) == 1, base
    for base in (2.0 ** -21, 0.5, 1.0, 3e38):
        assert f(base, 0) == 0, base         # no tokens: nothing runs
