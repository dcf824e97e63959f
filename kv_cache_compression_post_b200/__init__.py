"""kvb: historical KV-bank management (DensityKV, Forcing-KV), rotary positions and an 8-bit cache on sm_100a.

The binding lives in ``kv_cache_compression_post_b200.kvb`` (loaded on first
use: importing it fails loudly if ``libkvb.so`` has not been built with
``python -m kv_cache_compression_post_b200.build``).  Names such as
``kv_cache_compression_post_b200.kvb_admit`` are forwarded to it.
"""


def __getattr__(name):
    if name.startswith("kvb_") or name in ("KvbError", "make_config", "lib", "LIB_PATH", "Bank", "PAGES_PRESET",
                                            "Q8Cache", "rope") \
            or name.startswith("KVB_"):
        from . import kvb as _kvb
        value = globals()[name] = getattr(_kvb, name)   # found here from now on
        return value
    raise AttributeError(name)
