"""Host-side refusals of kvb_rope and the 8-bit cache's calls (no GPU: every check returns
before anything is launched)."""
import ctypes

import pytest

P = ctypes.c_void_p(0x10000)       # never dereferenced


def _cache(**kw):
    import kv_cache_compression_post_b200 as kvb
    f = dict(heads=2, head_dim=128, capacity=256, block=64, K=0x1000, V=0x2000, k_scale=0x3000, v_scale=0x4000,
             len=0x5000, mass=0x6000, status=0x7000)
    f.update(kw)
    return kvb.kvb_q8_cache(**f)


BAD_SIZES = [dict(heads=0), dict(heads=1025), dict(capacity=0), dict(capacity=-64), dict(capacity=100),
             dict(capacity=(1 << 24) + 64), dict(block=0), dict(block=48), dict(block=256)]
BAD_POINTERS = [dict(K=0), dict(V=0), dict(k_scale=0), dict(v_scale=0), dict(len=0), dict(K=0x1008), dict(V=0x2001),
                dict(k_scale=0x3002), dict(v_scale=0x4001), dict(len=0x5002), dict(mass=0x6001), dict(status=0x7003)]


def test_workspace_size():
    import kv_cache_compression_post_b200 as kvb
    base = kvb.kvb_q8_workspace_size(_cache(), 1, kvb.KVB_BF16)
    assert base > 0 and base % 256 == 0
    # an eviction of the whole capacity fits: one position per head and token
    assert kvb.kvb_q8_workspace_size(_cache(heads=1024, capacity=1 << 14), 1, kvb.KVB_BF16) >= 4 << 24
    assert kvb.kvb_q8_workspace_size(_cache(), 4680, kvb.KVB_BF16) >= base
    for kw in BAD_SIZES + [dict(head_dim=96), dict(head_dim=0)]:
        assert kvb.kvb_q8_workspace_size(_cache(**kw), 1, kvb.KVB_BF16) == 0, kw
    assert kvb.kvb_q8_workspace_size(_cache(), 0, kvb.KVB_BF16) == 0
    assert kvb.kvb_q8_workspace_size(_cache(), 1, 2) == 0
    assert kvb.lib.kvb_q8_workspace_size(None, 1, 0) == 0


def _calls(c):
    """One call of every entry point on this cache, otherwise valid."""
    import kv_cache_compression_post_b200 as kvb
    lib, r = kvb.lib, ctypes.byref(c)
    ws = ctypes.c_void_p(0x100000)
    other = ctypes.byref(_cache(K=0x11000, V=0x12000, k_scale=0x13000, v_scale=0x14000, len=0x15000, mass=0x16000))
    return [lib.kvb_q8_append(r, P, 128, 128, P, 128, 128, 4, 0, None, None),
            lib.kvb_q8_attend(r, P, 1, 0, 0.0, P, P, ws, 1 << 40, None),
            lib.kvb_q8_mass(r, P, 1, 0, 0.0, P, 1.0, None, ws, 1 << 40, None),
            lib.kvb_q8_evict(r, other, 8, 0, 0, None, ws, 1 << 40, None),
            lib.kvb_q8_evict(other, r, 8, 0, 0, None, ws, 1 << 40, None)]


@pytest.mark.parametrize("kw", BAD_SIZES + BAD_POINTERS, ids=str)
def test_every_call_refuses_a_bad_cache(kw):
    assert _calls(_cache(**kw)) == [1] * 5


@pytest.mark.parametrize("d", [0, 32, 96, 256])
def test_head_dims_without_a_kernel(d):
    assert _calls(_cache(head_dim=d)) == [7] * 5


def test_null_cache():
    import kv_cache_compression_post_b200 as kvb
    lib, c = kvb.lib, ctypes.byref(_cache())
    assert lib.kvb_q8_append(None, P, 128, 128, P, 128, 128, 4, 0, None, None) == 1
    assert lib.kvb_q8_attend(None, P, 1, 0, 0.0, P, P, P, 1 << 40, None) == 1
    assert lib.kvb_q8_mass(None, P, 1, 0, 0.0, P, 1.0, None, P, 1 << 40, None) == 1
    assert lib.kvb_q8_evict(None, c, 8, 0, 0, None, P, 1 << 40, None) == 1
    assert lib.kvb_q8_evict(c, None, 8, 0, 0, None, P, 1 << 40, None) == 1


def test_append_refusals():
    import kv_cache_compression_post_b200 as kvb
    f = kvb.lib.kvb_q8_append
    c = ctypes.byref(_cache())
    odd = ctypes.c_void_p(0x10008)
    assert f(c, P, 128, 128, P, 128, 128, -1, 0, None, None) == 1
    assert f(c, P, 128, 128, P, 128, 128, 257, 0, None, None) == 1           # more than the capacity
    assert f(c, P, 128, 128, P, 128, 128, 4, 2, None, None) == 1             # type
    assert f(c, None, 128, 128, P, 128, 128, 4, 0, None, None) == 1
    assert f(c, P, 128, 128, None, 128, 128, 4, 0, None, None) == 1
    assert f(c, odd, 128, 128, P, 128, 128, 4, 0, None, None) == 1
    assert f(c, P, 128, 128, odd, 128, 128, 4, 0, None, None) == 1
    for s in [(124, 128, 128, 128), (128, 124, 128, 128), (128, 128, 124, 128), (128, 128, 128, 124)]:
        assert f(c, P, s[0], s[1], P, s[2], s[3], 4, 0, None, None) == 1     # bf16 rows 8 bytes off
        assert f(c, P, s[0] + 2, s[1], P, s[2] + 2, s[3] + 2, 4, 1, None, None) == 1
    assert f(c, P, 128, 128, P, 128, 128, 4, 0, ctypes.c_void_p(0x5002), None) == 1
    for at in (0x5004, 0x4FFC):                                              # another head's length for a start
        assert f(c, P, 128, 128, P, 128, 128, 4, 0, ctypes.c_void_p(at), None) == 1
    assert f(c, None, 0, 0, None, 0, 0, 0, 0, None, None) == 0               # nothing to do


def test_attend_and_mass_refusals():
    import kv_cache_compression_post_b200 as kvb
    lib, c = kvb.lib, _cache()
    r, ws = ctypes.byref(c), ctypes.c_void_p(0x100000)
    need = kvb.kvb_q8_workspace_size(c, 33, 0)
    nan, inf, odd = float("nan"), float("inf"), ctypes.c_void_p(0x10008)
    att = lambda Q=P, n=33, t=0, s=0.0, O=P, l=P, w=ws, b=need: lib.kvb_q8_attend(r, Q, n, t, s, O, l, w, b, None)
    for kw, want in [(dict(Q=None), 1), (dict(O=None), 1), (dict(Q=odd), 1), (dict(O=odd), 1), (dict(n=0), 1),
                     (dict(n=-3), 1), (dict(t=2), 1), (dict(s=nan), 1), (dict(s=inf), 1), (dict(s=-1.0), 1),
                     (dict(l=ctypes.c_void_p(0x10002)), 1), (dict(w=None), 2), (dict(b=need - 1), 2),
                     (dict(w=ctypes.c_void_p(0x100080)), 2)]:
        assert att(**kw) == want, kw
    ms = lambda Q=P, n=33, t=0, s=0.0, l=P, d=1.0, p=None, w=ws, b=need: lib.kvb_q8_mass(r, Q, n, t, s, l, d, p, w, b, None)
    for kw, want in [(dict(Q=None), 1), (dict(l=None), 1), (dict(Q=odd), 1), (dict(n=0), 1), (dict(t=-1), 1),
                     (dict(s=nan), 1), (dict(d=nan), 1), (dict(d=inf), 1), (dict(p=ctypes.c_void_p(0x10001)), 1),
                     (dict(w=None), 2), (dict(b=need - 1), 2)]:
        assert ms(**kw) == want, kw
    bare = ctypes.byref(_cache(mass=0))
    assert lib.kvb_q8_mass(bare, P, 1, 0, 0.0, P, 1.0, None, ws, 1 << 40, None) == 1


def test_evict_refusals():
    import kv_cache_compression_post_b200 as kvb
    lib, ws = kvb.lib, ctypes.c_void_p(0x100000)
    to = dict(K=0x11000, V=0x12000, k_scale=0x13000, v_scale=0x14000, len=0x15000, mass=0x16000, capacity=128)
    need = kvb.kvb_q8_workspace_size(_cache(), 1, 0)

    def f(src=None, dst=None, budget=64, sink=4, recent=8, kept=None, w=ws, b=need):
        return lib.kvb_q8_evict(ctypes.byref(_cache(**(src or {}))), ctypes.byref(_cache(**{**to, **(dst or {})})), budget,
                                sink, recent, kept, w, b, None)

    for kw in [dict(budget=0), dict(budget=129), dict(sink=-1), dict(recent=-1), dict(sink=60, recent=5),
               dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(src=dict(mass=0)), dict(dst=dict(heads=3)),
               dict(dst=dict(head_dim=64)), dict(dst=dict(block=32)), dict(dst=dict(K=0x1000)), dict(dst=dict(V=0x2000)),
               dict(dst=dict(k_scale=0x3000)), dict(dst=dict(v_scale=0x4000)), dict(dst=dict(len=0x5000)),
               dict(dst=dict(mass=0x6000)), dict(kept=ctypes.c_void_p(0x10002))]:
        assert f(**kw) == 1, kw
    assert f(w=None) == 2 and f(b=need - 1) == 2 and f(w=ctypes.c_void_p(0x100010)) == 2


def test_rope_refusals():
    import kv_cache_compression_post_b200 as kvb
    odd, nan = ctypes.c_void_p(0x10008), float("nan")

    def f(X=P, pos=P, heads=2, n=5, d=64, t=0, pairs=(12, 10, 10), base=1e4, pairing=0, xs=(320, 64), out=P,
          os=(320, 64)):
        arr = None if pairs is None else (ctypes.c_int32 * 3)(*pairs)
        return kvb.lib.kvb_rope(X, pos, heads, n, d, t, arr, base, pairing, 0, xs[0], xs[1], out, os[0], os[1], None)

    for kw in [dict(X=None), dict(pos=None), dict(out=None), dict(X=odd), dict(out=odd), dict(heads=0),
               dict(heads=65536), dict(n=-1), dict(d=0), dict(d=60), dict(d=264), dict(t=2), dict(pairs=None),
               dict(pairs=(-1, 2, 2)), dict(pairs=(12, 11, 10)), dict(pairs=(2 ** 31 - 1, 2 ** 31 - 1, 2)),
               dict(base=0.0), dict(base=-2.0), dict(base=nan), dict(base=float("inf")), dict(pairing=2),
               dict(xs=(324, 64)), dict(xs=(320, 68)), dict(os=(322, 64)), dict(os=(320, 66)),
               dict(xs=(64, 128), os=(320, 64)),                 # in place with other strides
               dict(os=(0, 64)), dict(os=(320, 0)), dict(os=(0, 0))]:        # rows of out on one another
        assert f(**kw) == 1, kw
    assert f(n=0) == 0


def test_struct_mirror_matches_the_header(tmp_path):
    """The ctypes kvb_q8_cache has the layout a C compiler gives the header's."""
    import os
    import shutil
    import subprocess
    import kv_cache_compression_post_b200 as kvb
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "q8.c"
    names = [n for n, _ in kvb.kvb_q8_cache._fields_]
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "kvb.h"\nint main(void) {\n'
                   '  printf("%zu\\n", sizeof(kvb_q8_cache));\n' +
                   "".join(f'  printf("%zu\\n", offsetof(kvb_q8_cache, {n}));\n' for n in names) + "  return 0;\n}\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(root, "include"),
                    str(src), "-o", str(tmp_path / "q8")], check=True)
    out = subprocess.run([str(tmp_path / "q8")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in out] == [ctypes.sizeof(kvb.kvb_q8_cache)] + [getattr(kvb.kvb_q8_cache, n).offset for n in names]


def test_binding_refuses_wrong_tensors():
    """The helpers check shapes, types and layouts before any pointer is taken (CPU tensors
    are refused too)."""
    import torch
    import kv_cache_compression_post_b200 as kvb
    x, pos = torch.zeros(2, 3, 64), torch.zeros(3, 3, dtype=torch.int32)
    for args in [(x, pos, x), (x.half(), pos, x.half()), (x[0], pos, x[0])]:
        with pytest.raises(kvb.KvbError) as e:
            kvb.rope(*args, (12, 10, 10))
        assert e.value.status == 1
