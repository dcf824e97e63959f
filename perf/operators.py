"""Workloads of the rotary, 8-bit cache and weight-eviction operators, with their plain forms.

Six kinds of case, each one pass through one entry point of the package:

* ``rope``    rotary positions over (time, row, column), forwards or backwards (``kvb_rope``);
* ``append``  tokens rounded to E4M3 with one scale per block of tokens and head (``kvb_q8_append``);
* ``attend``  softmax attention read straight from that cache (``kvb_q8_attend``);
* ``mass``    the attention weight every cached token receives, summed over queries (``kvb_q8_mass``);
* ``evict``   the cache cut to a budget by that weight, order kept (``kvb_q8_evict``).

With ``own`` false the operators run in elementary torch operations in 32 bits (angles in 64); with it
true they run through the package.  Shapes follow the synthetic workloads of ``kvgen``: 12 heads of
128, 1560-token frames at 480P and 8160 at 1080P, three frames per chunk.
"""
import math

import torch

own = False

LARGEST_PAIRS = 4 * 24480 * 65280      # query-key pairs of the largest listed case


# ---------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------
def listed():
    return [
        # a 480P chunk's queries as the projection writes them ([token][head]), turned head-major while rotating
        dict(name="rope_chunk_480", kind="rope", heads=12, tokens=4680, dim=128, dtype="bf16", halves=False,
             inverse=False, token_major_in=True, frame_w=52, frame=1560),
        # the gradient of a 1080P chunk's keys in training: the inverse rotation, back to [token][head]
        dict(name="rope_grad_1080_f32", kind="rope", heads=12, tokens=24480, dim=128, dtype="f32", halves=True,
             inverse=True, token_major_in=False, frame_w=120, frame=8160),
        # one new token into a block that is already part full
        dict(name="append_token", kind="append", heads=12, dim=128, block=64, start=14117, tokens=1, dtype="bf16"),
        # a finalised 480P chunk behind an odd number of tokens: the first and last block are shared
        dict(name="append_chunk_480", kind="append", heads=12, dim=128, block=64, start=9361, tokens=4680,
             dtype="bf16"),
        # single-token attention over [sink | history | window] of 480P: launch latency counts
        dict(name="attend_token", kind="attend", heads=12, rows=1, length=15600, ragged=False, dim=128, block=64,
             dtype="bf16"),
        # a long cache whose heads are each shared by 8 query heads, of differing lengths
        dict(name="attend_group_long", kind="attend", heads=8, rows=8, length=131072, ragged=True, dim=128,
             block=128, dtype="bf16"),
        # a 480P chunk's attention in one layer
        dict(name="attend_chunk_480", kind="attend", heads=12, rows=4680, length=15600, ragged=False, dim=128,
             block=64, dtype="bf16"),
        # a 1080P chunk; four heads, so that the plain form's scores fit
        dict(name="attend_chunk_1080", kind="attend", heads=4, rows=24480, length=65280, ragged=False, dim=128,
             block=64, dtype="bf16"),
        # the weights one token spreads over a 480P cache, in single precision
        dict(name="mass_token_f32", kind="mass", heads=12, rows=1, length=15600, ragged=False, dim=128, block=64,
             dtype="f32"),
        # the weights a whole 480P chunk spreads over the cache it attended
        dict(name="mass_chunk_480", kind="mass", heads=12, rows=4680, length=15600, ragged=False, dim=128,
             block=64, dtype="bf16"),
        # a 480P cache cut back to six frames: the sink frame and the last chunk stay
        dict(name="evict_480", kind="evict", heads=12, dim=128, block=64, length=14040, ragged=False, budget=9360,
             sink=1560, recent=4680),
        # a long cache of differing lengths cut to a quarter
        dict(name="evict_long", kind="evict", heads=8, dim=128, block=128, length=131072, ragged=True,
             budget=32768, sink=16, recent=1024),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "append", "attend", "attend", "mass", "evict"])
    dim = rng.choice([64, 128])
    block = rng.choice([16, 32, 64, 128])
    if kind == "rope":
        dim = rng.choice([64, 80, 96, 128, 256])
        heads = rng.randint(1, 40)
        tokens = _spread(rng, 1, 24480 * 12 * 128 // (heads * dim))
        frame_w = rng.randint(4, 120)
        return dict(kind="rope", heads=heads, tokens=tokens, dim=dim, dtype=rng.choice(["bf16", "f32"]),
                    halves=rng.random() < 0.5, inverse=rng.random() < 0.5, token_major_in=rng.random() < 0.5,
                    frame_w=frame_w, frame=frame_w * rng.randint(4, 68))
    if kind == "append":
        return dict(kind="append", heads=rng.randint(1, 32), dim=dim, block=block, start=rng.randint(0, 20000),
                    tokens=_spread(rng, 1, 8192), dtype=rng.choice(["bf16", "f32"]))
    if kind in ("attend", "mass"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        heads = rng.randint(1, 24)
        if dtype == "f32":
            rows, length = _spread(rng, 1, 256), _spread(rng, 1, 8192)
        elif rng.random() < 0.5:
            rows, length = rng.randint(1, 16), _spread(rng, 1, 131072)
        else:
            rows = _spread(rng, 17, 8192)
            length = _spread(rng, 1, min(65536, LARGEST_PAIRS // (heads * rows)))
        return dict(kind=kind, heads=heads, rows=rows, length=length, ragged=rng.random() < 0.5, dim=dim,
                    block=block, dtype=dtype)
    length = _spread(rng, 16, 131072)
    budget = rng.randint(max(1, length // 8), length)
    sink = rng.randint(0, budget // 4)
    return dict(kind="evict", heads=rng.randint(1, 12), dim=dim, block=block, length=length,
                ragged=rng.random() < 0.5, budget=budget, sink=sink, recent=rng.randint(0, budget // 2))


def _lengths(case):
    """Tokens held per head: all of `length`, or falling from it to about half over the heads."""
    n, heads = case["length"], case["heads"]
    return [n - (h * n) // (2 * heads) if case["ragged"] else n for h in range(heads)]


def _capacity(case, tokens):
    return -(-tokens // case["block"]) * case["block"]


def work(case):
    dim = case.get("dim", 0)
    size = 2 if case.get("dtype") == "bf16" else 4
    kind, heads = case["kind"], case["heads"]
    if kind == "rope":
        n = heads * case["tokens"] * dim
        return dict(bytes=2 * n * size + 12 * case["tokens"], flops=3 * n)
    if kind == "append":
        n = heads * case["tokens"] * dim
        return dict(bytes=2 * n * (size + 1), flops=4 * n)
    keys = sum(_lengths(case))
    scales = 4 * keys / case["block"]
    if kind == "attend":
        rows = heads * case["rows"]
        return dict(bytes=2 * (keys * dim + scales) + rows * (2 * dim * size + 4), flops=4 * case["rows"] * keys * dim)
    if kind == "mass":
        rows = heads * case["rows"]
        return dict(bytes=keys * (dim + 4) + scales + rows * (dim * size + 4), flops=2 * case["rows"] * keys * dim)
    kept = sum(min(n, case["budget"]) for n in _lengths(case))
    return dict(bytes=4 * keys + kept * (4 * dim + 8) + 4 * kept * 4 / case["block"], flops=2 * kept * dim)


# ---------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _axis_pairs(dim):
    """(time, row, column) pairs of a head: a sixth of the width for row and column each, the rest for time."""
    rc = dim // 6
    return dim // 2 - 2 * rc, rc, rc


def _cache(case, seed, tokens):
    """E4M3 codes and power-of-two block scales of normal keys and values, some blocks larger than others."""
    g = _generator(seed)
    heads, dim, block, cap = case["heads"], case["dim"], case["block"], _capacity(case, tokens)
    s = {}
    for name in ("K", "V"):
        x = torch.randn(heads, cap // block, block, dim, generator=g, device="cuda")
        size = torch.randint(0, 3, (heads, cap // block), generator=g, device="cuda")
        # codes near the top of the format (448 = 64 * 7, seven deviations); values of size 1, 1/2 or 1/4
        s[name] = (64 * x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).reshape(heads, cap, dim)
        s[name.lower() + "_scale"] = torch.exp2(-6.0 - size.float())
    return s


def prepare(case, seed):
    g = _generator(seed + 7919)
    s = {"case": case}
    heads = case["heads"]
    if case["kind"] == "rope":
        n, dim = case["tokens"], case["dim"]
        shape = (n, heads, dim) if case["token_major_in"] else (heads, n, dim)
        x = torch.randn(shape, generator=g, device="cuda").to(_dtype(case))
        s["X"] = x.transpose(0, 1) if case["token_major_in"] else x             # [head][token][dim] views
        y = torch.empty((heads, n, dim) if case["token_major_in"] else (n, heads, dim), device="cuda",
                        dtype=_dtype(case))
        s["out"] = y if case["token_major_in"] else y.transpose(0, 1)
        i = torch.arange(n, device="cuda")
        first = int(torch.randint(0, 4096, (1,), generator=g, device="cuda"))
        at = i % case["frame"]
        s["pos"] = torch.stack([first + i // case["frame"], at // case["frame_w"], at % case["frame_w"]],
                               1).to(torch.int32).contiguous()
        s["pairs"] = _axis_pairs(dim)
        return s
    if case["kind"] == "append":
        tokens = case["start"] + case["tokens"]
        s.update(_cache(case, seed, tokens))
        shape = (case["tokens"], heads, case["dim"])
        # keys head-major (they were rotated), values as the projection writes them
        s["newK"] = torch.randn((heads, case["tokens"], case["dim"]), generator=g, device="cuda").to(_dtype(case))
        s["newV"] = torch.randn(shape, generator=g, device="cuda").to(_dtype(case)).transpose(0, 1)
        s["start"] = torch.full((heads,), case["start"], dtype=torch.int32, device="cuda")
        s["len"] = s["start"].clone()
        s["mass"] = None
    else:
        s.update(_cache(case, seed, case["length"]))
        s["len"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        s["mass"] = None
    if case["kind"] in ("attend", "mass"):
        shape = (heads, case["rows"], case["dim"])
        s["Q"] = (1.5 * torch.randn(shape, generator=g, device="cuda")).to(_dtype(case))
        s["scale"] = 1.0 / math.sqrt(case["dim"])
    if case["kind"] == "attend":
        s["O"] = torch.empty_like(s["Q"])
        s["lse"] = torch.empty(shape[:2], device="cuda")
    if case["kind"] == "mass":
        s["lse"] = _scores(s).logsumexp(-1)
        s["prev"] = torch.rand((heads, s["K"].shape[1]), generator=g, device="cuda")
        s["mass"] = torch.zeros_like(s["prev"])
    if case["kind"] == "evict":
        # accumulated weight: positive, with a long tail, and some exact ties
        w = torch.rand((heads, s["K"].shape[1]), generator=g, device="cuda")
        s["mass"] = torch.where(w < 0.02, torch.full_like(w, 0.5), (w + 1e-6) ** -0.5)
        cap = _capacity(case, case["budget"])
        for name in ("K", "V"):
            s["to" + name] = torch.zeros((heads, cap, case["dim"]), dtype=torch.uint8, device="cuda")
            s["to_%s_scale" % name.lower()] = torch.ones((heads, cap // case["block"]), device="cuda")
        s["to_mass"] = torch.zeros((heads, cap), device="cuda")
        s["to_len"] = torch.zeros(heads, dtype=torch.int32, device="cuda")
        s["kept"] = torch.full((heads, case["budget"]), -1, dtype=torch.int32, device="cuda")
    if own:
        import kv_cache_compression_post_b200 as kvb
        dtype = kvb.KVB_F32 if case.get("dtype") == "f32" else kvb.KVB_BF16
        s["cache"] = kvb.Q8Cache(heads, case["dim"], s["K"].shape[1], case["block"], dtype=dtype,
                                 max_queries=case.get("rows", 1), K=s["K"], V=s["V"], k_scale=s["k_scale"],
                                 v_scale=s["v_scale"], len=s["len"], mass=s["mass"])
        if case["kind"] == "evict":
            s["to"] = kvb.Q8Cache(heads, case["dim"], s["toK"].shape[1], case["block"], K=s["toK"], V=s["toV"],
                                  k_scale=s["to_k_scale"], v_scale=s["to_v_scale"], len=s["to_len"],
                                  mass=s["to_mass"])
    return s


# ---------------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------------
def run(s):
    kind = s["case"]["kind"]
    if own:
        return _own[kind](s)
    return _plain[kind](s)


def _own_rope(s):
    import kv_cache_compression_post_b200 as kvb
    c = s["case"]
    kvb.rope(s["X"], s["pos"], s["out"], s["pairs"],
             pairing=kvb.KVB_ROPE_HALVES if c["halves"] else kvb.KVB_ROPE_INTERLEAVED, inverse=c["inverse"])
    return s["out"]


def _own_append(s):
    s["cache"].append(s["newK"], s["newV"], start=s["start"])
    return _codes(s, s["K"], s["V"], s["k_scale"], s["v_scale"])


def _own_attend(s):
    s["cache"].attend(s["Q"], s["O"], s["lse"])
    return s["O"], s["lse"]


def _own_mass(s):
    s["cache"].accumulate(s["Q"], s["lse"], decay=0.875, prev=s["prev"])
    return s["mass"]


def _own_evict(s):
    c = s["case"]
    s["cache"].evict(s["to"], c["budget"], sink=c["sink"], recent=c["recent"], kept=s["kept"])
    return (s["kept"], s["to_len"], s["toK"].view(torch.float8_e4m3fn), s["toV"].view(torch.float8_e4m3fn),
            s["to_k_scale"], s["to_v_scale"], s["to_mass"])


_own = dict(rope=_own_rope, append=_own_append, attend=_own_attend, mass=_own_mass, evict=_own_evict)


def _rotation(s, wide):
    """cos and sin of every (token, pair), the angles in 64 bits."""
    c = s["case"]
    per = []
    for a, n in enumerate(s["pairs"]):
        f = 10000.0 ** (-torch.arange(n, dtype=torch.float64, device="cuda") / max(n, 1))
        per.append(s["pos"][:, a, None].double() * f)
    ang = torch.cat(per, 1)
    if c["inverse"]:
        ang = -ang
    return ang.cos().to(wide), ang.sin().to(wide)


def _plain_rope(s):
    c = s["case"]
    cos, sin = _rotation(s, torch.float32)
    x = s["X"].float()
    half = c["dim"] // 2
    a, b = (x[..., :half], x[..., half:]) if c["halves"] else (x[..., 0::2], x[..., 1::2])
    p, q = a * cos - b * sin, a * sin + b * cos
    return (torch.cat([p, q], -1) if c["halves"] else torch.stack([p, q], -1).flatten(-2)).to(s["X"].dtype)


def _codes(s, K, V, k_scale, v_scale):
    """The blocks that an append touched: codes as E4M3 values, and their scales."""
    c = s["case"]
    b0 = c["start"] // c["block"]
    at, end = b0 * c["block"], c["start"] + c["tokens"]
    return (K[:, at:end].view(torch.float8_e4m3fn), V[:, at:end].view(torch.float8_e4m3fn), k_scale[:, b0:],
            v_scale[:, b0:])


def _scale_of(amax):
    """The smallest power of two s with amax / s <= 448."""
    m, e = torch.frexp(amax)                                     # amax = m 2^e, 0.5 <= m < 1
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-100, 119)    # 448 = 0.875 * 2^9
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.full_like(amax, 2.0 ** -100))


def _plain_append(s):
    c = s["case"]
    block, start, n = c["block"], c["start"], c["tokens"]
    b0 = start // block
    nb = s["K"].shape[1] // block - b0
    out = []
    for codes, scale, new in ((s["K"], s["k_scale"], s["newK"]), (s["V"], s["v_scale"], s["newV"])):
        old = start - b0 * block                                  # tokens the first block already holds
        x = torch.zeros(c["heads"], nb * block, c["dim"], device="cuda")
        x[:, old:old + n] = new.float()
        amax = x.view(c["heads"], nb, block * c["dim"]).abs().amax(-1)
        sc = _scale_of(amax)
        if old:
            sc[:, 0] = torch.maximum(sc[:, 0], scale[:, b0])
            held = codes[:, start - old:start].view(torch.float8_e4m3fn).float()
            x[:, :old] = held * scale[:, b0, None, None]
        q = x.view(c["heads"], nb, block, c["dim"]) / sc[..., None, None]
        out.append((q.reshape(c["heads"], nb * block, c["dim"])[:, :old + n].to(torch.float8_e4m3fn), sc))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _values(codes, scale, block, wide=torch.float32):
    heads, cap, dim = codes.shape
    x = codes.view(torch.float8_e4m3fn).to(wide).view(heads, cap // block, block, dim)
    return (x * scale[..., None, None].to(wide)).view(heads, cap, dim)


def _scores(s):
    """Scaled scores [head][row][token], -inf past each head's length."""
    block = s["case"]["block"]
    S = (s["Q"].float() * s["scale"]) @ _values(s["K"], s["k_scale"], block).transpose(1, 2)
    past = torch.arange(S.shape[2], device="cuda") >= s["len"][:, None, None]
    return S.masked_fill_(past, -math.inf)


def _plain_attend(s):
    S = _scores(s)
    m = S.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    P = S.sub_(m).exp_()
    l = P.sum(-1, keepdim=True)
    O = P @ _values(s["V"], s["v_scale"], s["case"]["block"])
    O = torch.where(l > 0, O / l, torch.zeros_like(O))
    return O.to(s["Q"].dtype), (m + l.log())[..., 0]


def _plain_mass(s):
    w = _scores(s).sub_(s["lse"][..., None]).exp_().sum(1)
    held = torch.arange(w.shape[1], device="cuda") < s["len"][:, None]
    return torch.where(held, 0.875 * s["prev"] + w, torch.zeros_like(w))


def _plain_evict(s):
    c = s["case"]
    heads, budget, block, n = c["heads"], c["budget"], c["block"], s["len"].long()[:, None]
    at = torch.arange(s["mass"].shape[1], device="cuda")[None]
    # what must stay ranks before every weight, what is not held behind it
    rank = s["mass"].masked_fill((at < c["sink"]) | (at >= n - c["recent"]), math.inf)
    rank = rank.masked_fill(at >= n, -math.inf)
    order = rank.sort(dim=1, descending=True, stable=True)[1][:, :budget]
    left = torch.minimum(n, torch.full_like(n, budget))
    slot = torch.arange(budget, device="cuda")[None]
    order = torch.where(slot < left, order, torch.full_like(order, 1 << 40)).sort(1)[0]
    held = slot < left
    kept = torch.where(held, order, torch.full_like(order, -1))
    src = kept.clamp(min=0)
    cap = s["toK"].shape[1]
    pad = torch.nn.functional.pad
    outs = []
    for codes, scale in ((s["K"], s["k_scale"]), (s["V"], s["v_scale"])):
        sc = torch.where(held, scale.gather(1, src // block), torch.zeros_like(scale[:, :1]))
        to = pad(sc, (0, cap - budget)).view(heads, cap // block, block).amax(-1)
        each = pad(sc, (0, cap - budget)) / torch.where(to > 0, to, torch.ones_like(to)).repeat_interleave(block, 1)
        x = codes.view(torch.float8_e4m3fn).float().gather(1, src[..., None].expand(-1, -1, c["dim"]))
        x = pad(x, (0, 0, 0, cap - budget)) * each[..., None]
        outs.append((x.to(torch.float8_e4m3fn), torch.where(to > 0, to, torch.ones_like(to))))
    mass = pad(torch.where(held, s["mass"].gather(1, src), torch.zeros_like(s["mass"][:, :1])), (0, cap - budget))
    return (kept.int(), left[:, 0].int(), outs[0][0], outs[1][0], outs[0][1], outs[1][1], mass)


_plain = dict(rope=_plain_rope, append=_plain_append, attend=_plain_attend, mass=_plain_mass, evict=_plain_evict)


# ---------------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------------
def _nearest_e4m3(x):
    """The E4M3 value nearest to each x (ties to the even mantissa): steps of 2^(e-3) in [2^e, 2^(e+1)), e >= -6."""
    step = torch.exp2(torch.log2(x.abs().clamp(min=2.0 ** -6)).floor() - 3)
    return (x / step).round() * step


def _exact_append(s):
    c, out = s["case"], []
    first = c["start"] // c["block"]
    for codes, scale, new in (("K", "k_scale", "newK"), ("V", "v_scale", "newV")):
        old = s[codes][:, first * c["block"]:c["start"]].view(torch.float8_e4m3fn).double()
        old = old * s[scale][:, first, None, None].double()
        x, got, scales = torch.cat([old, s[new].double()], 1), [], []
        for i, part in enumerate(x.split(c["block"], 1)):
            fresh = part[:, old.shape[1]:] if i == 0 else part
            sc = torch.exp2((fresh.abs().amax((1, 2)) / 448).log2().ceil())
            if i == 0 and old.shape[1]:
                sc = torch.maximum(sc, s[scale][:, first].double())
            got.append(_nearest_e4m3(part / sc[:, None, None]))
            scales.append(sc)
        out.append((torch.cat(got, 1), torch.stack(scales, 1)))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _exact_evict(s):
    c, cap = s["case"], s["toK"].shape[1]
    kept = torch.full((c["heads"], c["budget"]), -1, dtype=torch.int32, device="cuda")
    wide = dict(dtype=torch.float64, device="cuda")
    mass, left = torch.zeros((c["heads"], cap), **wide), []
    code = {n: torch.zeros((c["heads"], cap, c["dim"]), **wide) for n in "KV"}
    to = {n: torch.ones((c["heads"], cap // c["block"]), **wide) for n in "KV"}
    for h in range(c["heads"]):
        n = int(s["len"][h])
        keep = list(range(n))
        if n > c["budget"]:
            w = s["mass"][h, :n].tolist()
            middle = sorted(range(c["sink"], n - c["recent"]), key=lambda i: (-w[i], i))
            middle = middle[:c["budget"] - c["sink"] - c["recent"]]
            keep = sorted(list(range(c["sink"])) + middle + list(range(n - c["recent"], n)))
        left.append(len(keep))
        at = torch.tensor(keep, device="cuda")
        kept[h, :len(keep)] = at.int()
        mass[h, :len(keep)] = s["mass"][h, at].double()
        for name, scales in (("K", "k_scale"), ("V", "v_scale")):
            each = s[scales][h].double()[at // c["block"]]
            for i, part in enumerate(each.split(c["block"])):
                to[name][h, i] = part.max()
            x = s[name][h, at].view(torch.float8_e4m3fn).double() * each[:, None]
            own_scale = to[name][h].repeat_interleave(c["block"])[:len(keep), None]
            code[name][h, :len(keep)] = _nearest_e4m3(x / own_scale)
    return (kept, torch.tensor(left, dtype=torch.int32), code["K"], code["V"], to["K"], to["V"], mass)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "rope":
        # each pair as one complex number times exp(i angle)
        x, half = s["X"].double(), case["dim"] // 2
        z = torch.complex(x[..., :half], x[..., half:]) if case["halves"] else torch.complex(x[..., 0::2], x[..., 1::2])
        angle = torch.empty(case["tokens"], half, dtype=torch.float64, device="cuda")
        k = 0
        for axis, n in enumerate(s["pairs"]):
            for j in range(n):
                angle[:, k] = s["pos"][:, axis].double() * math.pow(10000.0, -j / n)
                k += 1
        z = z * torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)
        return torch.cat([z.real, z.imag], -1) if case["halves"] else torch.view_as_real(z).flatten(-2)
    if kind == "append":
        return _exact_append(s)
    if kind == "evict":
        return _exact_evict(s)
    O, lse, mass = [], [], []
    for h in range(case["heads"]):
        n = int(s["len"][h])
        part = []
        for codes, scale in ((s["K"], s["k_scale"]), (s["V"], s["v_scale"])):
            x = codes[h, :n].view(torch.float8_e4m3fn).double()
            part.append(x * scale[h].double().repeat_interleave(case["block"])[:n, None])
        K, V = part
        w = torch.zeros(n, dtype=torch.float64, device="cuda")
        for r in range(0, case["rows"], 4096):
            q = s["Q"][h, r:r + 4096].double()
            S = q @ K.T / math.sqrt(case["dim"])
            if kind == "mass":
                w += torch.exp(S - s["lse"][h, r:r + 4096, None].double()).sum(0)
                continue
            z = torch.logsumexp(S, 1)
            O.append(torch.exp(S - z[:, None]) @ V)
            lse.append(z)
        if kind == "mass":
            full = torch.zeros(s["mass"].shape[1], dtype=torch.float64, device="cuda")
            full[:n] = w + 0.875 * s["prev"][h, :n].double()
            mass.append(full)
    if kind == "mass":
        return torch.stack(mass)
    return torch.cat(O).view(s["Q"].shape), torch.cat(lse).view(s["lse"].shape)
