"""What the 8-bit cache path is measured on: rotary positions, the append that
applies them, single-token attention and prompt attention, each in its plain
form (elementary torch, 32 bits) and through the library's entry points.

The cache (pool kind KV_POOL_FP8) holds e4m3 codes and one power-of-two scale
2^e per 16 tokens, KV head and tensor; a value is code * 2^e.  Stored order:
codes [page][head][tile of 16 tokens][K, V][2048]
  K byte (t, c): (t / 8) * 1024 + (c / 64) * 512 + (t % 8) * 64 + c % 64
  V byte (t, c): (t % 2 + 2 * (t / 8)) * 512 + (c / 16) * 64 + ((t % 8) / 2) * 16 + c % 16
exponents [page][head][tile][K, V] int8.
"""

import math

import numpy as np
import torch

own = False

D = 128            # head size
TILE = 16          # tokens that share a scale
E_MIN, E_MAX = -64, 7
LOG2E = 1.4426950408889634


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    half = {"style": "half", "rotary_dim": 128, "theta": 1e6, "scaling": "none", "factor": 1.0}
    yarn = {"style": "half", "rotary_dim": 128, "theta": 1e6, "scaling": "yarn", "factor": 4.0}
    part = {"style": "interleaved", "rotary_dim": 64, "theta": 1e4, "scaling": "linear", "factor": 2.0}
    return [
        # one new token for each of 64 sequences, q and k out of a fused projection
        {"name": "rope 64 tokens", "op": "rope", "tokens": 64, "hq": 32, "hkv": 8, "far": 32768, **half},
        # a prompt of 8192 tokens, half of each head rotated, neighbouring pairs
        {"name": "rope 8192 tokens", "op": "rope", "tokens": 8192, "hq": 64, "hkv": 8, "far": 131072, **part},
        # one decode step of a batch: 64 sequences at 8k to 32k tokens take one token each
        {"name": "append 64 x 1", "op": "append", "seqs": 64, "lo": 1, "hi": 1, "start_lo": 8192, "start_hi": 32768,
         "hq": 32, "hkv": 8, "page": 16, "shape": 1, **half},
        # a ragged batch of chunks that continue partly filled pages, positions scaled for long contexts
        {"name": "append 16 x 1-1000", "op": "append", "seqs": 16, "lo": 1, "hi": 1000, "start_lo": 0,
         "start_hi": 100000, "hq": 64, "hkv": 8, "page": 32, "shape": 2, **yarn},
        # a whole prompt of 8192 tokens into an empty cache
        {"name": "append 1 x 8192", "op": "append", "seqs": 1, "lo": 8192, "hi": 8192, "start_lo": 0, "start_hi": 0,
         "hq": 32, "hkv": 8, "page": 16, "shape": 3, **half},
        # the smallest decode of the benchmark's shapes: one sequence, 1024 tokens
        {"name": "decode 1 x 1024", "op": "decode", "seqs": 1, "lo": 1024, "hi": 1024, "hq": 8, "hkv": 2, "page": 16,
         "window": 0, "sinks": 0, "shape": 4},
        # one sequence at 100,000 tokens: the work is split over the cache
        {"name": "decode 1 x 100000", "op": "decode", "seqs": 1, "lo": 100000, "hi": 100000, "hq": 32, "hkv": 8,
         "page": 16, "window": 0, "sinks": 0, "shape": 5},
        # a served batch: 64 sequences of 8k to 32k tokens
        {"name": "decode 64 x 8k-32k", "op": "decode", "seqs": 64, "lo": 8192, "hi": 32768, "hq": 32, "hkv": 8,
         "page": 16, "window": 0, "sinks": 0, "shape": 6},
        # long contexts under a sliding window of 4096 tokens with 64 first tokens kept
        {"name": "decode 16 x 131072 window", "op": "decode", "seqs": 16, "lo": 131072, "hi": 131072, "hq": 64,
         "hkv": 8, "page": 32, "window": 4096, "sinks": 64, "shape": 7},
        # a short prompt
        {"name": "prefill 1 x 512", "op": "prefill", "seqs": 1, "lo": 512, "hi": 512, "prefix_lo": 0, "prefix_hi": 0,
         "hq": 32, "hkv": 8, "page": 16, "window": 0, "sinks": 0, "shape": 8},
        # ragged chunks on cached prefixes under a sliding window with 64 first tokens kept
        {"name": "prefill 4 x 300-2000 window", "op": "prefill", "seqs": 4, "lo": 300, "hi": 2000, "prefix_lo": 1000,
         "prefix_hi": 12000, "hq": 64, "hkv": 8, "page": 32, "window": 4096, "sinks": 64, "shape": 9},
        # a prompt of 8192 tokens, all of it visible
        {"name": "prefill 1 x 8192", "op": "prefill", "seqs": 1, "lo": 8192, "hi": 8192, "prefix_lo": 0,
         "prefix_hi": 0, "hq": 32, "hkv": 8, "page": 16, "window": 0, "sinks": 0, "shape": 10},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv = rng.choice([(8, 2), (32, 8), (64, 8), (8, 8), (16, 8), (8, 1), (40, 10)])
    page, shape = rng.choice([16, 32]), rng.randrange(1 << 30)
    op = rng.choice(["rope", "append", "decode", "prefill"])
    rope = {"style": rng.choice(["half", "interleaved"]), "rotary_dim": rng.choice([32, 64, 96, 128]),
            "theta": rng.choice([1e4, 5e5, 1e6]), "scaling": rng.choice(["none", "linear", "ntk", "yarn"]),
            "factor": rng.choice([2.0, 4.0, 8.0])}
    if op == "rope":
        return {"op": op, "tokens": _log(rng, 1, 8192), "hq": hq, "hkv": hkv, "far": _log(rng, 64, 1000000), **rope}
    if op == "append":
        hi = _log(rng, 1, 8192)
        lo = rng.choice([hi, max(1, hi // 3), 1])
        far = _log(rng, 1, 100000)
        return {"op": op, "seqs": min(_log(rng, 1, 64), max(1, 8192 // hi)), "lo": lo, "hi": hi,
                "start_lo": rng.choice([0, far]), "start_hi": far, "hq": hq, "hkv": hkv, "page": page,
                "shape": shape, **rope}
    window = rng.choice([0, _log(rng, 16, 8192)])
    sinks = rng.choice([0, rng.randrange(1, 129)])
    if op == "decode":
        hi = _log(rng, 1, 131072)
        seqs = min(_log(rng, 1, 64), max(1, (8 << 20) // (hi * hkv)))
        return {"op": op, "seqs": seqs, "lo": rng.choice([hi, max(1, hi // 4), 0]), "hi": hi, "hq": hq, "hkv": hkv,
                "page": page, "window": window, "sinks": sinks, "shape": shape}
    hi = _log(rng, 2, 4096)
    far = _log(rng, 1, 32768)
    seqs = min(_log(rng, 1, 8), max(1, 2 ** 30 // (hq * hi * (hi + far))))
    while hq * hi * (hi + far) > 2 ** 30:
        far, hi = far // 2, max(2, hi * 3 // 4)
    return {"op": op, "seqs": seqs, "lo": rng.choice([hi, max(1, hi // 3)]), "hi": hi, "prefix_lo": 0,
            "prefix_hi": far, "hq": hq, "hkv": hkv, "page": page, "window": window, "sinks": sinks, "shape": shape}


def _shape(case):
    """Lengths and page table of a case: int64 arrays `n` (new tokens or queries), `start`
    (tokens before them), and the pages, shuffled.  An append's earlier pages are not held:
    only those that it writes are."""
    g = np.random.default_rng(case["shape"])
    b, p = case["seqs"], case["page"]
    n = g.integers(case["lo"], case["hi"] + 1, b)
    n[0] = case["hi"]
    if case["op"] == "append":
        start = g.integers(case["start_lo"], case["start_hi"] + 1, b)
        first = start // p
    elif case["op"] == "prefill":
        start = g.integers(case["prefix_lo"], case["prefix_hi"] + 1, b)
        first = np.zeros(b, np.int64)
    else:
        start, first = n - 1, np.zeros(b, np.int64)
    end = start + n if case["op"] != "decode" else n
    last = (end + p - 1) // p
    width = max(1, int(last.max()))
    held = (np.arange(width) >= first[:, None]) & (np.arange(width) < last[:, None])
    pages = int(held.sum()) + 1
    table = np.zeros((b, width), np.int32)
    table[held] = g.permutation(pages)[:int(held.sum())]
    return n, start, end, table, pages


def _seen(case, pos):
    """How many keys a query at position `pos` (array) attends to."""
    w, s = case["window"], case["sinks"]
    total = np.maximum(pos + 1, 0)
    if not w:
        return total
    return np.minimum(total, np.minimum(total, w) + np.minimum(s, np.maximum(total - w, 0)))


def work(case):
    hq, hkv = case["hq"], case["hkv"]
    row = 2 * D                                     # one bf16 row
    if case["op"] == "rope":
        t = case["tokens"]
        return {"bytes": 2 * t * (hq + hkv) * row + 4 * t, "flops": 3 * t * (hq + hkv) * case["rotary_dim"]}
    n, start, end, table, pages = _shape(case)
    if case["op"] == "append":
        t = int(n.sum())
        tiles = int(((end + TILE - 1) // TILE - start // TILE).sum())
        return {"bytes": t * (2 * hq + 2 * hkv) * row + t * hkv * 2 * D + 2 * tiles * hkv,
                "flops": 3 * t * (hq + hkv) * case["rotary_dim"] + 4 * t * hkv * D}
    if case["op"] == "decode":
        keys = int(_seen(case, n - 1).sum())
        b = len(n)
        return {"bytes": keys * hkv * 2 * D + keys // TILE * hkv * 2 + 2 * b * hq * row + 4 * b * hq,
                "flops": 4 * keys * hq * D}
    pairs = sum(int(_seen(case, np.arange(s, e)).sum()) for s, e in zip(start, end))
    first = [min(int(e), case["sinks"] + case["window"] + int(m) - 1) if case["window"] else int(e)
             for m, e in zip(n, end)]
    t = int(n.sum())
    return {"bytes": sum(first) * hkv * 2 * D + 2 * t * hq * row + 4 * t * hq, "flops": 4 * pairs * hq * D}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _inv_freq(case):
    """Rotation speeds in radians per position [rotary_dim / 2] (64 bits) and the factor on
    cos and sin."""
    d, base, f = case["rotary_dim"], case["theta"], case["factor"]
    i = np.arange(d // 2)
    if case["scaling"] == "ntk":
        base = base * f ** (d / (d - 2))
    w = base ** (-2.0 * i / d)
    if case["scaling"] == "linear":
        return w / f, 1.0
    if case["scaling"] == "yarn":
        dim = lambda turns: d * math.log(32768 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), d - 1)
        ramp = np.clip((i - low) / max(high - low, 0.001), 0.0, 1.0)
        return w / f * ramp + w * (1.0 - ramp), 0.1 * math.log(f) + 1.0
    return w, 1.0


def _cache(case, pages, g):
    """Stored codes and exponents as a cache holds them: N(0, 1) values, a few channels larger."""
    tiles = case["page"] // TILE
    shape = (pages, case["hkv"], tiles, 2, TILE * D)
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat = codes.view(-1)
    for lo in range(0, flat.numel(), 1 << 28):
        part = torch.randn(min(1 << 28, flat.numel() - lo), generator=g, device="cuda").mul_(100.0)
        flat[lo:lo + part.numel()] = part.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    exps = torch.randint(-8, -5, shape[:4], generator=g, device="cuda").to(torch.int8)
    return codes, exps


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    hq, hkv = case["hq"], case["hkv"]
    s = dict(case)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    i32 = lambda a: torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    if "scaling" in case:
        inv, s["att"] = _inv_freq(case)
        s["inv_freq"] = torch.as_tensor(inv).cuda()
    if case["op"] == "rope":
        t, pages, seqs = case["tokens"], 1, 1
        s["qkv"] = randn(t, hq + 2 * hkv, D)
        s["pos"] = torch.randint(0, case["far"], (t,), generator=g, device="cuda").to(torch.int32)
        s["out"] = [torch.empty(t, h, D, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv)]
    else:
        n, start, end, table, pages = _shape(case)
        seqs, t = case["seqs"], int(n.sum())
        s["n"], s["start"], s["end"] = i32(n), i32(start), i32(end)
        s["table"], s["width"], s["total"] = i32(table), table.shape[1], t
        s["cu"] = i32(np.concatenate([[0], np.cumsum(n)]))
        s["most"], s["longest"] = int(n.max()), int(end.max())
        s["codes"], s["exps"] = _cache(case, pages, g)
        if case["op"] == "append":
            s["qkv"] = randn(t, hq + 2 * hkv, D)
            s["qkv"][:, hq:, ::37] *= 4
            s["out"] = torch.empty(t, hq, D, dtype=torch.bfloat16, device="cuda")
        else:
            rows = seqs if case["op"] == "decode" else t
            s["q"] = randn(rows, hq, D)
            s["out"] = torch.empty(rows, hq, D, dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.empty(rows, hq, dtype=torch.float32, device="cuda")
            s["scale"] = 1.0 / math.sqrt(D)
    if own:
        from bit_kv_cache_12_gb300 import native
        page = case.get("page", 16)
        pool = native.KVPool(native.KV_POOL_FP8, 1, hq, hkv, page, pages, seqs)
        s["pool"] = pool
        if "scaling" in case:
            native.kv_pool_set_rope(pool.handle, 0, native.rope_config(
                rotary_dim=case["rotary_dim"], style=case["style"], theta=case["theta"], scaling=case["scaling"],
                factor=case["factor"], original_max_position=32768))
        if "codes" in s:
            codes, exps = pool.fp8_views(0)
            codes.copy_(s["codes"])
            exps.copy_(s["exps"])
            s["codes"], s["exps"] = codes, exps
        if case["op"] == "decode":
            s["ws_bytes"] = native.kv_decode_workspace_bytes(pool.handle, seqs, s["longest"])
        if case["op"] == "prefill":
            s["ws_bytes"] = native.kv_prefill_workspace_bytes(pool.handle, seqs, s["most"], s["longest"])
        if "ws_bytes" in s:
            s["ws"] = torch.empty(max(16, s["ws_bytes"]), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _RUN_OWN[s["op"]](s)
    return _RUN_PLAIN[s["op"]](s)


def _own_rope(s):
    from bit_kv_cache_12_gb300 import native
    hq, hkv, qkv = s["hq"], s["hkv"], s["qkv"]
    row = qkv.stride(0)
    native.kv_rope_apply(s["pool"].handle, 0, s["tokens"], s["pos"], qkv, row, qkv[:, hq:], row, s["out"][0], hq * D,
                         s["out"][1], hkv * D)
    return s["out"]


def _own_append(s):
    from bit_kv_cache_12_gb300 import native
    hq, hkv, qkv = s["hq"], s["hkv"], s["qkv"]
    row = qkv.stride(0)
    native.kv_append_fp8(s["pool"].handle, 0, s["seqs"], qkv, row, qkv[:, hq:], row, qkv[:, hq + hkv:], row, s["cu"],
                         s["start"], s["table"], s["width"], s["most"], s["out"])
    return {"q": s["out"], "codes": s["codes"].view(torch.float8_e4m3fn), "exps": s["exps"]}


def _own_decode(s):
    from bit_kv_cache_12_gb300 import native
    native.kv_decode_attention_fp8(s["pool"].handle, 0, s["seqs"], s["q"], s["end"], s["table"], s["width"],
                                   s["longest"], s["scale"], s["window"], s["sinks"], s["out"], s["lse"], s["ws"],
                                   s["ws_bytes"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_prefill(s):
    from bit_kv_cache_12_gb300 import native
    native.kv_prefill_attention_fp8(s["pool"].handle, 0, s["seqs"], s["q"], s["cu"], s["end"], s["table"], s["width"],
                                    s["most"], s["longest"], s["scale"], s["window"], s["sinks"], s["out"], s["lse"],
                                    s["ws"], s["ws_bytes"])
    return {"out": s["out"], "lse": s["lse"]}


_RUN_OWN = {"rope": _own_rope, "append": _own_append, "decode": _own_decode, "prefill": _own_prefill}


# ---- plain forms ------------------------------------------------------------

def _rotated(x, pos, s):
    """x [T, H, D] (any type) rotated by its positions, in 32 bits; angles in 64."""
    angle = pos.double()[:, None] * s["inv_freq"]
    cos = (torch.cos(angle) * s["att"]).float()[:, None]
    sin = (torch.sin(angle) * s["att"]).float()[:, None]
    r = s["rotary_dim"]
    y = x.float()
    part = y[..., :r]
    if s["style"] == "half":
        a, b = part[..., :r // 2], part[..., r // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., r:]], -1)


def _plain_rope(s):
    hq, hkv, qkv = s["hq"], s["hkv"], s["qkv"]
    return [_rotated(qkv[:, :hq], s["pos"], s).to(torch.bfloat16),
            _rotated(qkv[:, hq:hq + hkv], s["pos"], s).to(torch.bfloat16)]


def _k_order(x):
    """[..., 16, 128] token rows -> [..., 2048] stored K order."""
    return x.unflatten(-1, (2, 64)).unflatten(-3, (2, 8)).transpose(-3, -2).flatten(-4)


def _v_order(x):
    """[..., 16, 128] token rows -> [..., 2048] stored V order."""
    n = x.dim() - 2
    y = x.unflatten(-1, (8, 16)).unflatten(n, (2, 4, 2))         # t / 8, t % 8 / 2, t % 2, c / 16, c % 16
    return y.permute(*range(n), n, n + 2, n + 3, n + 1, n + 4).flatten(n)


def _k_rows(x):
    """[..., 2048] stored K order -> [..., 16, 128] token rows."""
    return x.unflatten(-1, (2, 2, 8, 64)).transpose(-3, -2).flatten(-2).flatten(-3, -2)


def _v_rows(x):
    """[..., 2048] stored V order -> [..., 16, 128] token rows."""
    n = x.dim() - 1
    y = x.unflatten(-1, (2, 2, 8, 4, 16))            # t / 8, t % 2, c / 16, t % 8 / 2, c % 16
    return y.permute(*range(n), n, n + 3, n + 1, n + 2, n + 4).flatten(-2).flatten(-4, -2)


def _pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _exponent(square):
    """The smallest e with square <= (448 * 2^e)^2, within the cache's range."""
    f, x = torch.frexp(square)
    e = torch.div(x - 18 + (f > 0.765625).int() + 1, 2, rounding_mode="floor")
    e = torch.where(square > 0, e, E_MIN)
    return torch.where(torch.isinf(square), E_MAX, e).clamp(E_MIN, E_MAX).int()


def _plain_append(s):
    hq, hkv, qkv, p = s["hq"], s["hkv"], s["qkv"], s["page"]
    t = s["total"]
    seq = torch.repeat_interleave(torch.arange(s["seqs"], device="cuda"), s["n"].long(), output_size=t)
    pos = s["start"].long()[seq] + torch.arange(t, device="cuda") - s["cu"].long()[seq]
    q = _rotated(qkv[:, :hq], pos, s).to(torch.bfloat16)
    raw_k, v = qkv[:, hq:hq + hkv].float(), qkv[:, hq + hkv:].float()
    k = _rotated(raw_k, pos, s)
    # a pair's length does not change under rotation: the K scale goes by it
    r, att2 = s["rotary_dim"], float(np.float32(s["att"])) ** 2
    sq = raw_k * raw_k
    a, b = ((sq[..., :r // 2], sq[..., r // 2:r]) if s["style"] == "half" else (sq[..., 0:r:2], sq[..., 1:r:2]))
    pairs = a + b
    if att2 != 1.0:
        pairs = pairs * torch.tensor(att2, dtype=torch.float32, device="cuda")
    size = torch.stack([torch.cat([pairs, sq[..., r:]], -1).amax(-1), (v * v).amax(-1)], -1)     # [t, hkv, 2]
    # one entry per (page, tile of the page) that is written
    slot = pos % p
    where = s["table"].long()[seq, pos // p] * (p // TILE) + slot // TILE
    tile, back = torch.unique(where, return_inverse=True)
    most = torch.zeros(tile.numel(), hkv, 2, device="cuda")
    most = most.scatter_reduce(0, back[:, None, None].expand(-1, hkv, 2), size, "amax")
    first = torch.full((tile.numel(),), TILE, device="cuda").scatter_reduce(0, back, slot % TILE, "amin")
    at = (tile // (p // TILE), slice(None), tile % (p // TILE))
    e_old = s["exps"][at].int()                                                                   # [n, hkv, 2]
    e_new = _exponent(most)
    e_new = torch.where((first > 0)[:, None, None], torch.maximum(e_new, e_old), e_new)
    # what the tile holds: earlier tokens moved to the new scale, later ones as they are
    held = s["codes"][at]                                                                         # [n, hkv, 2, 2048]
    rows = torch.stack([_k_rows(held[:, :, 0]), _v_rows(held[:, :, 1])], 2)                       # [n, hkv, 2, 16, 128]
    moved = rows.view(torch.float8_e4m3fn).float() * _pow2(e_old - e_new)[..., None, None]
    moved = moved.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    early = torch.arange(TILE, device="cuda") < first[:, None]
    rows = torch.where(early[:, None, None, :, None], moved, rows)
    new = torch.stack([k, v], 2) * _pow2(-e_new)[back][..., None]                                 # [t, hkv, 2, 128]
    rows[back, :, :, slot % TILE] = new.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s["codes"][at] = torch.stack([_k_order(rows[:, :, 0]), _v_order(rows[:, :, 1])], 2)
    s["exps"][at] = e_new.to(torch.int8)
    return {"q": q, "codes": s["codes"].view(torch.float8_e4m3fn), "exps": s["exps"]}


def _gathered(s, tiles):
    """K and V of tile indexes [B, n] as fp32 [B, hkv, n * 16, 128]."""
    per = s["page"] // TILE
    page = torch.gather(s["table"].long(), 1, (tiles // per).clamp(max=s["width"] - 1))
    codes, exps = s["codes"][page, :, tiles % per], s["exps"][page, :, tiles % per]
    scale = _pow2(exps.int())
    k = _k_rows(codes[:, :, :, 0]).view(torch.float8_e4m3fn).float() * scale[..., 0, None, None]
    v = _v_rows(codes[:, :, :, 1]).view(torch.float8_e4m3fn).float() * scale[..., 1, None, None]
    return [x.transpose(1, 2).flatten(2, 3) for x in (k, v)]


def _softmax_rows(logits, seen, v):
    """Softmax of logits [..., r, n] over the places of `seen`, times v [..., n, 128], and its log-sum-exp."""
    logits = logits.masked_fill_(~seen, -math.inf)
    top = logits.amax(-1, keepdim=True)
    base = torch.where(torch.isinf(top), 0.0, top)
    p = logits.sub_(base).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return out, (base + torch.log(total)).squeeze(-1)


def _plain_decode(s):
    b, hq, hkv, w, sinks = s["seqs"], s["hq"], s["hkv"], s["window"], s["sinks"]
    length = s["end"].long()
    every = torch.arange((s["longest"] + TILE - 1) // TILE, device="cuda").expand(b, -1)
    if w and w + sinks + 3 * TILE < s["longest"]:     # the tiles of the first tokens and of the window
        front = (sinks + TILE - 1) // TILE
        low = ((length - w).clamp(min=0) // TILE).clamp(min=front)
        every = torch.cat([every[:, :front], low[:, None] + torch.arange(w // TILE + 2, device="cuda")], 1)
    every = every.contiguous()
    k, v = _gathered(s, every)
    pos = (every[:, :, None] * TILE + torch.arange(TILE, device="cuda")).flatten(1)
    seen = pos < length[:, None]
    if w:
        seen = seen & ((pos >= length[:, None] - w) | (pos < sinks))
    q = s["q"].float().unflatten(1, (hkv, hq // hkv)) * s["scale"]
    out, lse = _softmax_rows(torch.matmul(q, k.transpose(-1, -2)), seen[:, None, None], v)
    return {"out": out.flatten(1, 2).to(torch.bfloat16), "lse": lse.flatten(1)}


def _plain_prefill(s):
    b, hq, hkv, w, sinks, most = s["seqs"], s["hq"], s["hkv"], s["window"], s["sinks"], s["most"]
    every = torch.arange((s["longest"] + TILE - 1) // TILE, device="cuda").expand(b, -1).contiguous()
    k, v = _gathered(s, every)
    key = torch.arange(every.shape[1] * TILE, device="cuda")
    row = torch.arange(most, device="cuda")
    live = row < s["n"][:, None]                                                                  # [b, most]
    pos = s["start"][:, None] + row
    seen = (key <= pos[..., None]) & live[..., None]
    if w:
        seen = seen & ((key > pos[..., None] - w) | (key < sinks))
    index = (s["cu"][:-1, None] + row).clamp(max=s["total"] - 1).long()
    q = s["q"][index].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4) * s["scale"]  # [b, hkv, g, most, D]
    logits = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (hq // hkv, most))
    out, lse = _softmax_rows(logits, seen[:, None, None], v[:, :, None])
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)                                                # [b, most, hq, D]
    lse = lse.permute(0, 3, 1, 2).flatten(2, 3)
    return {"out": out[live].to(torch.bfloat16), "lse": lse[live]}


_RUN_PLAIN = {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"rope": _exact_rope, "append": _exact_append, "decode": _exact_decode, "prefill": _exact_prefill}[
        case["op"]](case, s)


def _turn64(x, pos, case):
    """Pairs as complex numbers, multiplied by att * exp(i * pos * w)."""
    w, att = _inv_freq(case)
    x = x.double().clone()
    r = case["rotary_dim"]
    one = slice(0, r // 2) if case["style"] == "half" else slice(0, r, 2)
    two = slice(r // 2, r) if case["style"] == "half" else slice(1, r, 2)
    angle = pos.double()[:, None, None] * torch.as_tensor(w, device=x.device)
    z = torch.complex(x[..., one], x[..., two]) * torch.polar(torch.full_like(angle, att), angle)
    x[..., one], x[..., two] = z.real, z.imag
    return x


def _exact_rope(case, s):
    hq, hkv = case["hq"], case["hkv"]
    return [_turn64(s["qkv"][:, :hq], s["pos"], case), _turn64(s["qkv"][:, hq:hq + hkv], s["pos"], case)]


def _table64():
    """The 256 values of e4m3, from its definition."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append((-x if c & 128 else x) if c & 127 != 127 else math.nan)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _round64(x):
    """The nearest e4m3 value of each x, ties to even, the largest 448."""
    step = torch.exp2(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1].double() - 4)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _places():
    """Stored positions of (token, channel) in a tile: K and V, int64 [16, 128]."""
    t, c = np.meshgrid(np.arange(TILE), np.arange(D), indexing="ij")
    k = t // 8 * 1024 + c // 64 * 512 + t % 8 * 64 + c % 64
    v = (t % 2 + t // 8 * 2) * 512 + c // 16 * 64 + t % 8 // 2 * 16 + c % 16
    return [torch.as_tensor(x).cuda() for x in (k, v)]


def _exact_append(case, s):
    hq, hkv, p = case["hq"], case["hkv"], case["page"]
    n, start, end, table, pages = _shape(case)
    x = s["qkv"].double()
    at = torch.as_tensor(np.concatenate([np.arange(a, b) for a, b in zip(start, end)])).cuda()
    q = _turn64(x[:, :hq], at, case)
    rows = [_turn64(x[:, hq:hq + hkv], at, case), x[:, hq + hkv:]]
    r, att = case["rotary_dim"], _inv_freq(case)[1]
    k0 = x[:, hq:hq + hkv]
    one, two = ((k0[..., :r // 2], k0[..., r // 2:r]) if case["style"] == "half" else (k0[..., 0:r:2], k0[..., 1:r:2]))
    size = [torch.cat([torch.hypot(one, two) * att, k0[..., r:].abs()], -1).amax(-1), rows[1].abs().amax(-1)]
    values = _table64()[s["codes"].long()]
    exps = s["exps"].clone()
    places, row0 = _places(), 0
    for b in range(case["seqs"]):
        for tile in range(int(start[b]) // TILE, (int(end[b]) + TILE - 1) // TILE):
            lo, hi = max(int(start[b]), tile * TILE), min(int(end[b]), tile * TILE + TILE)
            new = slice(row0 + lo - int(start[b]), row0 + hi - int(start[b]))
            page, sub, first = int(table[b, tile * TILE // p]), tile % (p // TILE), lo % TILE
            for kv, place in enumerate(places):
                big = size[kv][new].amax(0)
                e = torch.ceil(torch.log2(big / 448))
                e = torch.where(big <= 448 * torch.exp2(e - 1), e - 1, e).clamp(E_MIN, E_MAX)
                cell = values[page, :, sub, kv]
                if first:
                    old = exps[page, :, sub, kv].double()
                    e = torch.maximum(e, old)
                    early = place[:first].flatten()
                    cell[:, early] = _round64(cell[:, early] * torch.exp2(old - e)[:, None])
                into = place[first:first + hi - lo].flatten()
                cell[:, into] = _round64(rows[kv][new] * torch.exp2(-e)[None, :, None]).transpose(0, 1).flatten(1)
                exps[page, :, sub, kv] = e.to(torch.int8)
        row0 += int(n[b])
    return {"q": q, "codes": values, "exps": exps}


def _sequence64(case, s, b, length):
    """K and V of one sequence: [hkv, length, 128] in 64 bits."""
    p = case["page"]
    pages = s["table"][b, :(length + p - 1) // p].long()
    table = _table64()
    got = []
    for kv, place in enumerate(_places()):
        x = table[s["codes"][pages][:, :, :, kv].long()][..., place]                  # [pages, hkv, tiles, 16, 128]
        x = x * torch.exp2(s["exps"][pages][:, :, :, kv].double())[..., None, None]
        got.append(x.transpose(0, 1).flatten(1, 3)[:, :length])
    return got


def _attend64(case, q, k, v, pos):
    """q [t, g, 128] of one KV head at positions pos [t] over k, v [n, 128]."""
    x = torch.einsum("tgd,nd->tgn", q.double(), k) / math.sqrt(D)
    key = torch.arange(k.shape[0], device=k.device)
    hide = key > pos[:, None]
    if case["window"]:
        hide = hide | ((key <= pos[:, None] - case["window"]) & (key >= case["sinks"]))
    x = x.masked_fill_(hide[:, None], -math.inf)
    lse = torch.logsumexp(x, -1)
    return torch.einsum("tgn,nd->tgd", torch.exp(x - lse[..., None]), v), lse


def _exact_rows(case, s, spans):
    hq, hkv = case["hq"], case["hkv"]
    g = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, (row, count, length) in enumerate(spans):
        if length <= 0 or count <= 0:
            continue
        k, v = _sequence64(case, s, b, length)
        pos = torch.arange(length - count, length, device="cuda")
        for h in range(hkv):
            heads = slice(h * g, h * g + g)
            out[row:row + count, heads], lse[row:row + count, heads] = _attend64(
                case, s["q"][row:row + count, heads], k[h], v[h], pos)
    return {"out": out, "lse": lse}


def _exact_decode(case, s):
    n = _shape(case)[0]
    return _exact_rows(case, s, [(b, 1 if m else 0, int(m)) for b, m in enumerate(n)])


def _exact_prefill(case, s):
    n, start, end, table, pages = _shape(case)
    row = np.concatenate([[0], np.cumsum(n)])
    return _exact_rows(case, s, [(int(row[b]), int(n[b]), int(end[b])) for b in range(case["seqs"])])
