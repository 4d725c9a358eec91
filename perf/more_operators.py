"""What the 4-bit cache path is measured on: rotary positions with several axes, writing
tokens into the cache and reading them back, single-token attention over it, and causal
attention over packed prompts of bf16 rows, each in its plain form (elementary torch,
32 bits) and through the library's entry points.

The cache (pool kind KV_POOL_FP4) holds e2m1 codes and one e4m3 scale per token, KV head,
tensor and block of 16 channels; a value is code * scale * 2^e, e one exponent per layer
and tensor.  A tile is 16 tokens of one KV head, 2304 bytes, tokens t and channels c at
  K code  64 t + c / 2, in the low four bits where c is even
  V code  1024 + 512 (c / 64) + 64 ((c % 16) / 2) + 16 ((t % 8) / 2) + 4 ((c / 16) % 4)
          + 2 (t / 8) + c % 2, in the low four bits where t is even
  K scale 2048 + 8 t + c / 16
  V scale 2176 + 32 ((t % 8) / 2) + 4 (c / 16) + 2 (t / 8) + t % 2
and the cache is [page][head][tile of the page][2304].
"""

import math

import numpy as np
import torch

own = False

D = 128            # head size
TILE = 16          # tokens of a tile
BLOCK = 16         # channels that share a scale
TILE_BYTES = 2304
V_CODES, K_SCALES, V_SCALES = 1024, 2048, 2176
ROW = 2 * D        # bytes of a bf16 row


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    big = {"hq": 32, "hkv": 8, "page": 16}
    wide = {"hq": 64, "hkv": 8, "page": 32}
    return [
        # one new token for each of 64 sequences; q and k are parts of a fused projection
        {"name": "rope axes 64 tokens", "op": "rope", "tokens": 64, "axes": 3, "layout": "blocks", "style": "half",
         "rotary_dim": 128, "theta": 1e6, "far": 32768, "shape": 1, **big},
        # a prompt of 8192 tokens, text and images, the axes taking turns over the pairs
        {"name": "rope axes 8192 tokens", "op": "rope", "tokens": 8192, "axes": 3, "layout": "turns", "style": "half",
         "rotary_dim": 128, "theta": 1e6, "far": 8192, "shape": 2, **wide},
        # one decode step of a batch: 64 sequences at 8k to 32k tokens take one token each
        {"name": "store 64 x 1", "op": "store", "seqs": 64, "lo": 1, "hi": 1, "start_lo": 8192, "start_hi": 32768,
         "k_exp": 0, "v_exp": 0, "shape": 3, **big},
        # a whole prompt of 8192 tokens into an empty cache
        {"name": "store 1 x 8192", "op": "store", "seqs": 1, "lo": 8192, "hi": 8192, "start_lo": 0, "start_hi": 0,
         "k_exp": 0, "v_exp": 0, "shape": 4, **big},
        # a short cached prefix that a chunk continues
        {"name": "read 1 x 1000", "op": "read", "seqs": 1, "lo": 1000, "hi": 1000, "start_lo": 0, "start_hi": 0,
         "k_exp": 0, "v_exp": 0, "shape": 5, **big},
        # ragged cached prefixes of a batch of chunks
        {"name": "read 8 x 1000-12000", "op": "read", "seqs": 8, "lo": 1000, "hi": 12000, "start_lo": 0, "start_hi": 0,
         "k_exp": 2, "v_exp": -3, "shape": 6, **wide},
        # the smallest decode of the benchmark's shapes: one sequence, 1024 tokens
        {"name": "decode 1 x 1024", "op": "decode", "seqs": 1, "lo": 1024, "hi": 1024, "hq": 8, "hkv": 2, "page": 16,
         "window": 0, "sinks": 0, "k_exp": 0, "v_exp": 0, "shape": 7},
        # one sequence at 100,000 tokens: the work is split over the cache
        {"name": "decode 1 x 100000", "op": "decode", "seqs": 1, "lo": 100000, "hi": 100000, "window": 0, "sinks": 0,
         "k_exp": 0, "v_exp": 0, "shape": 8, **big},
        # a served batch: 64 sequences of 8k to 32k tokens
        {"name": "decode 64 x 8k-32k", "op": "decode", "seqs": 64, "lo": 8192, "hi": 32768, "window": 0, "sinks": 0,
         "k_exp": 0, "v_exp": 0, "shape": 9, **big},
        # a short prompt
        {"name": "prompt 1 x 512", "op": "prompt", "seqs": 1, "lo": 512, "hi": 512, "prefix_lo": 0, "prefix_hi": 0,
         "window": 0, "sinks": 0, "shape": 10, **big},
        # packed chunks of different lengths behind prefixes, under a sliding window with 64 first tokens kept
        {"name": "prompt 4 x 300-2000 window", "op": "prompt", "seqs": 4, "lo": 300, "hi": 2000, "prefix_lo": 1000,
         "prefix_hi": 12000, "window": 4096, "sinks": 64, "shape": 11, **wide},
        # a prompt of 8192 tokens, all of it visible
        {"name": "prompt 1 x 8192", "op": "prompt", "seqs": 1, "lo": 8192, "hi": 8192, "prefix_lo": 0, "prefix_hi": 0,
         "window": 0, "sinks": 0, "shape": 12, **big},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv = rng.choice([(8, 2), (32, 8), (64, 8), (8, 8), (16, 8), (8, 1), (40, 10)])
    c = {"op": rng.choice(["rope", "store", "read", "decode", "prompt"]), "hq": hq, "hkv": hkv,
         "page": rng.choice([16, 32]), "shape": rng.randrange(1 << 30)}
    if c["op"] == "rope":
        return {**c, "tokens": _log(rng, 1, 8192), "axes": rng.choice([2, 3, 4]), "layout": rng.choice(["blocks", "turns"]),
                "style": rng.choice(["half", "interleaved"]), "rotary_dim": rng.choice([32, 64, 96, 128]),
                "theta": rng.choice([1e4, 5e5, 1e6]), "far": _log(rng, 64, 1000000)}
    exps = {"k_exp": rng.choice([0, -4, 3]), "v_exp": rng.choice([0, -3, 2])}
    window = rng.choice([0, _log(rng, 16, 8192)])
    sinks = rng.choice([0, rng.randrange(1, 129)])
    if c["op"] in ("store", "read"):
        hi = _log(rng, 1, 8192)
        far = _log(rng, 1, 100000)
        return {**c, **exps, "seqs": min(_log(rng, 1, 64), max(1, 8192 // hi)), "lo": rng.choice([hi, max(1, hi // 3), 1]),
                "hi": hi, "start_lo": rng.choice([0, far]), "start_hi": far}
    if c["op"] == "decode":
        hi = _log(rng, 1, 131072)
        return {**c, **exps, "seqs": min(_log(rng, 1, 64), max(1, (8 << 20) // (hi * hkv))),
                "lo": rng.choice([hi, max(1, hi // 4), 0]), "hi": hi, "window": window, "sinks": sinks}
    hi = _log(rng, 2, 4096)
    far = rng.choice([0, _log(rng, 1, 32768)])
    seqs = min(_log(rng, 1, 8), max(1, 2 ** 30 // (hq * hi * (hi + far))))
    while hq * hi * (hi + far) > 2 ** 30:
        far, hi = far // 2, max(2, hi * 3 // 4)
    return {**c, "seqs": seqs, "lo": rng.choice([hi, max(1, hi // 3)]), "hi": hi, "prefix_lo": 0, "prefix_hi": far,
            "window": window, "sinks": sinks}


def _shape(case):
    """Lengths and page table of a case: int64 arrays `n` (new tokens, tokens read, or queries),
    `start` (tokens before them) and `end`, and the pages, shuffled.  Where tokens are stored or
    read, only the pages that hold them exist."""
    g = np.random.default_rng(case["shape"])
    b, p = case["seqs"], case["page"]
    n = g.integers(case["lo"], case["hi"] + 1, b)
    n[0] = case["hi"]
    if case["op"] in ("store", "read"):
        start = g.integers(case["start_lo"], case["start_hi"] + 1, b)
        first, end = start // p, start + n
    elif case["op"] == "prompt":
        start = g.integers(case["prefix_lo"], case["prefix_hi"] + 1, b)
        return n, start, start + n, None, 1
    else:
        start, first, end = n - 1, np.zeros(b, np.int64), n
    last = (end + p - 1) // p
    width = max(1, int(last.max()))
    held = (np.arange(width) >= first[:, None]) & (np.arange(width) < last[:, None])
    pages = int(held.sum()) + 1
    table = np.zeros((b, width), np.int32)
    table[held] = g.permutation(pages)[:int(held.sum())]
    return n, start, end, table, pages


def _axis(case):
    """Which axis turns each of the rotary_dim / 2 pairs: a quarter of them the first and the rest
    the others in blocks, or all in turns."""
    n, axes = case["rotary_dim"] // 2, case["axes"]
    if case["layout"] == "turns":
        return [i % axes for i in range(n)]
    first = n // 4
    return [0 if i < first else 1 + (i - first) * (axes - 1) // (n - first) for i in range(n)]


def _positions(case):
    """int32 [axes, tokens] of text runs (the same position on every axis) and image grids
    (the first axis stands, the last two count rows and columns)."""
    g = np.random.default_rng(case["shape"])
    t, axes = case["tokens"], case["axes"]
    out = np.zeros((axes, t), np.int64)
    at, pos = 0, int(g.integers(0, case["far"]))
    while at < t:
        if g.integers(2):
            n = min(t - at, int(g.integers(1, 200)))
            out[:, at:at + n] = pos + np.arange(n)
            pos += n
        else:
            rows, cols = int(g.integers(1, 40)), int(g.integers(1, 40))
            n = min(t - at, rows * cols)
            out[:, at:at + n] = pos
            out[axes - 2, at:at + n] += np.arange(n) // cols
            out[axes - 1, at:at + n] += np.arange(n) % cols
            pos += max(rows, cols)
        at += n
    return out.astype(np.int32)


def _seen(case, pos):
    """How many keys a query at position `pos` (array) attends to."""
    w, s = case["window"], case["sinks"]
    total = np.maximum(pos + 1, 0)
    if not w:
        return total
    return np.minimum(total, np.minimum(total, w) + np.minimum(s, np.maximum(total - w, 0)))


def work(case):
    hq, hkv = case["hq"], case["hkv"]
    stored = 2 * (D // 2 + D // BLOCK)               # bytes of a cached token and KV head
    if case["op"] == "rope":
        t = case["tokens"]
        return {"bytes": 2 * t * (hq + hkv) * ROW + 4 * case["axes"] * t, "flops": 3 * t * (hq + hkv) * case["rotary_dim"]}
    n, start, end, table, pages = _shape(case)
    t = int(n.sum())
    if case["op"] == "store":                        # rows in, codes and scales written, rows read back
        return {"bytes": t * hkv * (4 * ROW + stored), "flops": 8 * t * hkv * D}
    if case["op"] == "read":
        return {"bytes": t * hkv * (2 * ROW + stored), "flops": 4 * t * hkv * D}
    if case["op"] == "decode":
        keys = int(_seen(case, n - 1).sum())
        return {"bytes": keys * hkv * stored + 2 * len(n) * hq * ROW + 4 * len(n) * hq, "flops": 4 * keys * hq * D}
    pairs = sum(int(_seen(case, np.arange(s, e)).sum()) for s, e in zip(start, end))
    used = [min(int(e), case["sinks"] + case["window"] + int(m) - 1) if case["window"] else int(e) for m, e in zip(n, end)]
    return {"bytes": sum(used) * hkv * 2 * ROW + 2 * t * hq * ROW + 4 * t * hq, "flops": 4 * pairs * hq * D}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _cache(case, pages, g):
    """Stored tiles as quantised N(0, 1) rows give them, one block of K's channels four times as large."""
    tiles = pages * case["hkv"] * (case["page"] // TILE)
    cache = torch.empty(tiles, TILE_BYTES, dtype=torch.uint8, device="cuda")
    # eight random bits -> the e2m1 code of a normal value whose block's largest is about 6
    value = 2.9 * torch.special.ndtri((torch.arange(256, dtype=torch.float64) + 0.5) / 256)
    mag = torch.bucketize(value.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64))
    code = (mag + 8 * (value < 0)).to(torch.uint8).cuda()
    step = max(1, (1 << 27) // K_SCALES)
    for lo in range(0, tiles, step):
        part = cache[lo:lo + step]
        bits = torch.randint(0, 1 << 16, (part.shape[0], K_SCALES), generator=g, device="cuda", dtype=torch.int32)
        part[:, :K_SCALES] = code[bits & 255] | (code[bits >> 8] << 4)
        scale = 0.3 * torch.exp(0.15 * torch.randn(part.shape[0], TILE_BYTES - K_SCALES, generator=g, device="cuda"))
        scale[:, 3:V_SCALES - K_SCALES:D // BLOCK] *= 4
        part[:, K_SCALES:] = scale.to(torch.float8_e4m3fn).view(torch.uint8)
    return cache.view(pages, case["hkv"], case["page"] // TILE, TILE_BYTES)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    hq, hkv = case["hq"], case["hkv"]
    s = dict(case)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    i32 = lambda a: torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    empty = lambda *shape: torch.empty(*shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    pages, seqs = 1, case.get("seqs", 1)
    if case["op"] == "rope":
        t = case["tokens"]
        s["qkv"] = randn(t, hq + 2 * hkv, D)
        s["pos"] = i32(_positions(case))
        s["axis"] = _axis(case)
        s["out"] = [empty(t, hq, D), empty(t, hkv, D)]
    else:
        n, start, end, table, pages = _shape(case)
        t = s["total"] = int(n.sum())
        s["n"], s["start"], s["end"] = i32(n), i32(start), i32(end)
        s["cu"] = i32(np.concatenate([[0], np.cumsum(n)]))
        s["most"], s["longest"] = int(n.max()), int(end.max())
        s["scale"] = 1.0 / math.sqrt(D)
        if table is not None:
            s["table"], s["width"] = i32(table), table.shape[1]
            s["cache"] = _cache(case, pages, g)
        if case["op"] == "store":
            s["kv"] = randn(t, 2 * hkv, D)
            s["kv"][:, :hkv, 48:64] *= 4
        if case["op"] in ("store", "read"):
            s["out"] = {"k": empty(t, hkv, D), "v": empty(t, hkv, D)}
        if case["op"] == "prompt":
            s["cu_k"] = i32(np.concatenate([[0], np.cumsum(end)]))
            s["keys"] = int(end.sum())
            if s["keys"] == t:                       # whole prompts: parts of one projection
                qkv = randn(t, hq + 2 * hkv, D)
                s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
            else:                                    # chunks: keys and values of prefix and chunk together
                s["q"], s["k"], s["v"] = randn(t, hq, D), randn(s["keys"], hkv, D), randn(s["keys"], hkv, D)
        if case["op"] in ("decode", "prompt"):
            rows = seqs if case["op"] == "decode" else t
            if case["op"] == "decode":
                s["q"] = randn(rows, hq, D)
            s["out"] = empty(rows, hq, D)
            s["lse"] = torch.empty(rows, hq, dtype=torch.float32, device="cuda")
    if own:
        from bit_kv_cache_12_gb300 import native
        kind = native.KV_POOL_FP4 if "cache" in s else native.KV_POOL_BF16
        pool = s["pool"] = native.KVPool(kind, 1, hq, hkv, case["page"], pages, seqs)
        if case["op"] == "rope":
            native.kv_pool_set_rope(pool.handle, 0, native.rope_config(
                rotary_dim=case["rotary_dim"], style=case["style"], theta=case["theta"]))
            native.kv_pool_set_rope_axes(pool.handle, 0, case["axes"], s["axis"])
        if "cache" in s:
            native.kv_pool_set_fp4_range(pool.handle, 0, case["k_exp"], case["v_exp"])
            view = pool.fp4_view(0)
            view.copy_(s["cache"])
            s["cache"] = view
        if case["op"] == "decode":
            s["ws_bytes"] = native.kv_decode_workspace_bytes(pool.handle, seqs, s["longest"])
        if case["op"] == "prompt":
            s["ws_bytes"] = native.kv_prompt_workspace_bytes(pool.handle, seqs, s["most"], s["longest"])
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
    native.kv_rope_apply_axes(s["pool"].handle, 0, s["tokens"], s["pos"], s["tokens"], qkv, row, qkv[:, hq:], row,
                              s["out"][0], hq * D, s["out"][1], hkv * D)
    return s["out"]


def _own_store(s):
    from bit_kv_cache_12_gb300 import native
    kv, row = s["kv"], s["kv"].stride(0)
    native.kv_append_fp4(s["pool"].handle, 0, s["seqs"], kv, row, kv[:, s["hkv"]:], row, s["cu"], s["start"], s["table"],
                         s["width"], s["most"])
    return _own_read(s)


def _own_read(s):
    from bit_kv_cache_12_gb300 import native
    row = s["hkv"] * D
    native.kv_read_fp4(s["pool"].handle, 0, s["seqs"], s["cu"], s["start"], s["table"], s["width"], s["most"],
                       s["out"]["k"], row, s["out"]["v"], row)
    return s["out"]


def _own_decode(s):
    from bit_kv_cache_12_gb300 import native
    native.kv_decode_attention_fp4(s["pool"].handle, 0, s["seqs"], s["q"], s["end"], s["table"], s["width"],
                                   s["longest"], s["scale"], s["window"], s["sinks"], s["out"], s["lse"], s["ws"],
                                   s["ws_bytes"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_prompt(s):
    from bit_kv_cache_12_gb300 import native
    q, k, v = s["q"], s["k"], s["v"]
    native.kv_prompt_attention(s["pool"].handle, s["seqs"], q, q.stride(0), s["total"], k, k.stride(0), v, v.stride(0),
                               s["keys"], s["cu"], s["cu_k"], s["most"], s["longest"], s["scale"], s["window"],
                               s["sinks"], s["out"], s["lse"], s["ws"], s["ws_bytes"])
    return {"out": s["out"], "lse": s["lse"]}


_RUN_OWN = {"rope": _own_rope, "store": _own_store, "read": _own_read, "decode": _own_decode, "prompt": _own_prompt}


# ---- plain forms ------------------------------------------------------------

def _plain_rope(s):
    hq, hkv, qkv, r = s["hq"], s["hkv"], s["qkv"], s["rotary_dim"]
    speed = s["theta"] ** (-2.0 * torch.arange(r // 2, device="cuda", dtype=torch.float64) / r)
    angle = s["pos"][torch.tensor(s["axis"], device="cuda")].double().transpose(0, 1) * speed       # [t, r / 2]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    x = qkv[:, :hq + hkv].float()
    part = x[..., :r]
    if s["style"] == "half":
        a, b = part[..., :r // 2], part[..., r // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    y = torch.cat([turned, x[..., r:]], -1).to(torch.bfloat16)
    return [y[:, :hq].contiguous(), y[:, hq:].contiguous()]


def _blocks(x):
    """fp32 rows [..., 128] -> e2m1 values [..., 8, 16] as fp32 and their e4m3 scales [..., 8]."""
    x = x.unflatten(-1, (D // BLOCK, BLOCK))
    scale = (x.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = scale.float()[..., None]
    a = torch.where(d > 0, x.abs() / d, 0.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    return torch.where(x < 0, -a, a), scale


def _code(v):
    """e2m1 values -> four-bit codes (uint8)."""
    a = v.abs()
    mag = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4))
    return (mag + torch.where(v < 0, 8.0, 0.0)).to(torch.uint8)


def _value(c):
    """Four-bit codes -> e2m1 values in fp32."""
    return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")[c.int()]


def _codes_of(tiles):
    """Stored tiles [..., 2304] -> K and V codes, uint8 [..., 16, 128] each."""
    k = tiles[..., :V_CODES].unflatten(-1, (TILE, D // 2))
    k = torch.stack([k & 15, k >> 4], -1).flatten(-2)
    n = tiles.dim() - 1
    v = tiles[..., V_CODES:K_SCALES].unflatten(-1, (2, 8, 4, 4, 2, 2))       # c / 64, c % 16 / 2, t % 8 / 2, c / 16 % 4, t / 8, c % 2
    v = torch.stack([v & 15, v >> 4], -1)                                    # t % 2
    v = v.permute(*range(n), n + 4, n + 2, n + 6, n, n + 3, n + 1, n + 5)
    return k, v.flatten(-4).flatten(-4, -2)


def _scales_of(tiles):
    """Stored tiles -> K and V scales, uint8 [..., 16, 8] each."""
    n = tiles.dim() - 1
    k = tiles[..., K_SCALES:V_SCALES].unflatten(-1, (TILE, D // BLOCK))
    v = tiles[..., V_SCALES:].unflatten(-1, (4, D // BLOCK, 2, 2))           # t % 8 / 2, c / 16, t / 8, t % 2
    return k, v.permute(*range(n), n + 2, n, n + 3, n + 1).flatten(-4, -2)


def _tiles_of(codes, scales):
    """The other way."""
    n = codes[0].dim() - 2
    k = codes[0].unflatten(-1, (D // 2, 2))
    v = codes[1].unflatten(-1, (2, 4, 8, 2)).unflatten(-5, (2, 4, 2))        # t / 8, t % 8 / 2, t % 2, c / 64, c / 16 % 4, c % 16 / 2, c % 2
    v = v.permute(*range(n), n + 3, n + 5, n + 1, n + 4, n, n + 6, n + 2)
    vs = scales[1].unflatten(-2, (2, 4, 2)).permute(*range(n), n + 1, n + 3, n, n + 2)
    return torch.cat([(k[..., 0] | (k[..., 1] << 4)).flatten(-2), (v[..., 0] | (v[..., 1] << 4)).flatten(-6),
                      scales[0].flatten(-2), vs.flatten(-4)], -1)


def _rows_of(tiles, s):
    """Stored tiles -> K and V rows, fp32 [..., 16, 128] each."""
    got = []
    for code, scale, e in zip(_codes_of(tiles), _scales_of(tiles), (s["k_exp"], s["v_exp"])):
        d = scale.view(torch.float8_e4m3fn).float() * 2.0 ** e
        got.append((_value(code).unflatten(-1, (D // BLOCK, BLOCK)) * d[..., None]).flatten(-2))
    return got


def _places(s):
    """Where each token of a store or read case is: its tile (flat index into pages and tiles of a
    page) and its slot there."""
    t, p = s["total"], s["page"]
    seq = torch.repeat_interleave(torch.arange(s["seqs"], device="cuda"), s["n"].long(), output_size=t)
    pos = s["start"].long()[seq] + torch.arange(t, device="cuda") - s["cu"].long()[seq]
    return s["table"].long()[seq, pos // p] * (p // TILE) + pos % p // TILE, pos % TILE


def _plain_store(s):
    hkv, per = s["hkv"], s["page"] // TILE
    where, slot = _places(s)
    tile, back = torch.unique(where, return_inverse=True)
    at = (tile // per, slice(None), tile % per)
    held = s["cache"][at]                                                    # [tiles, hkv, 2304]
    codes, scales = _codes_of(held), [x.clone() for x in _scales_of(held)]
    codes = [x.clone() for x in codes]
    for w, (part, e) in enumerate(((s["kv"][:, :hkv], s["k_exp"]), (s["kv"][:, hkv:], s["v_exp"]))):
        value, scale = _blocks(part.float() * 2.0 ** -e)
        codes[w][back, :, slot] = _code(value.flatten(-2))
        scales[w][back, :, slot] = scale.view(torch.uint8)
    s["cache"][at] = _tiles_of(codes, scales)
    return _plain_read(s)


def _plain_read(s):
    where, slot = _places(s)
    per = s["page"] // TILE
    tile, back = torch.unique(where, return_inverse=True)
    rows = _rows_of(s["cache"][tile // per, :, tile % per], s)               # [tiles, hkv, 16, 128]
    return {"k": rows[0][back, :, slot].to(torch.bfloat16), "v": rows[1][back, :, slot].to(torch.bfloat16)}


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
    b, hq, hkv, w, sinks, per = s["seqs"], s["hq"], s["hkv"], s["window"], s["sinks"], s["page"] // TILE
    length = s["end"].long()
    every = torch.arange((s["longest"] + TILE - 1) // TILE, device="cuda").expand(b, -1)
    if w and w + sinks + 3 * TILE < s["longest"]:     # the tiles of the first tokens and of the window
        front = (sinks + TILE - 1) // TILE
        low = ((length - w).clamp(min=0) // TILE).clamp(min=front)
        every = torch.cat([every[:, :front], low[:, None] + torch.arange(w // TILE + 2, device="cuda")], 1)
    every = every.contiguous()
    page = torch.gather(s["table"].long(), 1, (every // per).clamp(max=s["width"] - 1))
    k, v = [x.transpose(1, 2).flatten(2, 3) for x in _rows_of(s["cache"][page, :, every % per], s)]
    pos = (every[:, :, None] * TILE + torch.arange(TILE, device="cuda")).flatten(1)
    seen = pos < length[:, None]
    if w:
        seen = seen & ((pos >= length[:, None] - w) | (pos < sinks))
    q = s["q"].float().unflatten(1, (hkv, hq // hkv)) * s["scale"]
    out, lse = _softmax_rows(torch.matmul(q, k.transpose(-1, -2)), seen[:, None, None], v)
    return {"out": out.flatten(1, 2).to(torch.bfloat16), "lse": lse.flatten(1)}


def _plain_prompt(s):
    b, hq, hkv, w, sinks, most = s["seqs"], s["hq"], s["hkv"], s["window"], s["sinks"], s["most"]
    key = torch.arange(s["longest"], device="cuda")
    row = torch.arange(most, device="cuda")
    at = (s["cu_k"][:-1, None].long() + key).clamp(max=s["keys"] - 1)                             # [b, longest]
    k, v = s["k"][at].float().transpose(1, 2), s["v"][at].float().transpose(1, 2)                 # [b, hkv, longest, D]
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


_RUN_PLAIN = {"rope": _plain_rope, "store": _plain_store, "read": _plain_read, "decode": _plain_decode,
              "prompt": _plain_prompt}


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
    return {"rope": _exact_rope, "store": _exact_store, "read": _exact_read, "decode": _exact_decode,
            "prompt": _exact_prompt}[case["op"]](case, s)


def _exact_rope(case, s):
    """Pairs as complex numbers, multiplied by exp(i * position * speed)."""
    hq, hkv, r = case["hq"], case["hkv"], case["rotary_dim"]
    x = s["qkv"][:, :hq + hkv].double()
    first, second = (range(0, r // 2), range(r // 2, r)) if case["style"] == "half" else (range(0, r, 2), range(1, r, 2))
    for pair, (a, b) in enumerate(zip(first, second)):
        turn = s["pos"][s["axis"][pair]].double() * case["theta"] ** (-2.0 * pair / r)
        z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(turn), turn)[:, None]
        x[..., a], x[..., b] = z.real, z.imag
    return [x[:, :hq], x[:, hq:]]


def _nearest64(x, values):
    """The nearest of `values` (ascending, from 0) to each |x|; halfway, the one at an even place."""
    values = torch.tensor(values, dtype=torch.float64, device=x.device)
    mid = (values[1:] + values[:-1]) / 2
    a = x.abs().contiguous()
    up, down = torch.bucketize(a, mid, right=True), torch.bucketize(a, mid)
    return torch.copysign(values[torch.where(up % 2 == 0, up, down)], x)


def _e4m3_64():
    return [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127]


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_store(case, s):
    got = {}
    for name, x, e in (("k", s["kv"][:, :case["hkv"]], case["k_exp"]), ("v", s["kv"][:, case["hkv"]:], case["v_exp"])):
        x = (x.double() * 2.0 ** -e).unflatten(-1, (-1, BLOCK))
        scale = _nearest64(x.abs().amax(-1, keepdim=True) / 6, _e4m3_64())
        code = torch.where(scale > 0, _nearest64(x / torch.where(scale > 0, scale, 1.0), E2M1), 0.0)
        got[name] = (code * scale).flatten(-2) * 2.0 ** e
    return got


def _sequence64(case, s, b, lo, hi):
    """K and V of tokens [lo, hi) of one sequence: [hkv, hi - lo, 128] in 64 bits."""
    p = case["page"]
    pos = torch.arange(lo, hi, device="cuda")
    tile = s["cache"][s["table"][b].long()[pos // p], :, pos % p // TILE]                         # [n, hkv, 2304]
    t, c = (pos % TILE)[:, None], torch.arange(D, device="cuda")
    at = [(64 * t + c // 2, c % 2 + 0 * t, K_SCALES + 8 * t + c // 16),
          (V_CODES + 512 * (c // 64) + 64 * (c % 16 // 2) + 16 * (t % 8 // 2) + 4 * (c // 16 % 4) + 2 * (t // 8) + c % 2,
           t % 2 + 0 * c, V_SCALES + 32 * (t % 8 // 2) + 4 * (c // 16) + 2 * (t // 8) + t % 2)]
    code64 = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64, device="cuda")
    scale64 = torch.tensor(_e4m3_64() + [math.nan], dtype=torch.float64, device="cuda")
    got = []
    for (where, high, scale), e in zip(at, (case["k_exp"], case["v_exp"])):
        spread = lambda i: i[:, None].expand(-1, case["hkv"], -1)  # noqa: E731
        byte = torch.gather(tile, 2, spread(where)).int()
        code = torch.where(spread(high) == 1, byte >> 4, byte & 15)
        x = code64[code.long()] * scale64[torch.gather(tile, 2, spread(scale)).long()] * 2.0 ** e
        got.append(x.transpose(0, 1))
    return got


def _exact_read(case, s):
    n, start, end, table, pages = _shape(case)
    rows = [_sequence64(case, s, b, int(lo), int(hi)) for b, (lo, hi) in enumerate(zip(start, end))]
    return {name: torch.cat([r[w].transpose(0, 1) for r in rows]) for w, name in enumerate(("k", "v"))}


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


def _exact_rows(case, s, spans, keys_of):
    hq, hkv = case["hq"], case["hkv"]
    g = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, (row, count, length) in enumerate(spans):
        if length <= 0 or count <= 0:
            continue
        k, v = keys_of(b, length)
        pos = torch.arange(length - count, length, device="cuda")
        for h in range(hkv):
            heads = slice(h * g, h * g + g)
            out[row:row + count, heads], lse[row:row + count, heads] = _attend64(
                case, s["q"][row:row + count, heads], k[h], v[h], pos)
    return {"out": out, "lse": lse}


def _exact_decode(case, s):
    n = _shape(case)[0]
    return _exact_rows(case, s, [(b, 1 if m else 0, int(m)) for b, m in enumerate(n)],
                       lambda b, length: _sequence64(case, s, b, 0, length))


def _exact_prompt(case, s):
    n, start, end, table, pages = _shape(case)
    row, first = np.concatenate([[0], np.cumsum(n)]), np.concatenate([[0], np.cumsum(end)])
    keys = lambda b, length: [x[int(first[b]):int(first[b]) + length].double().transpose(0, 1)  # noqa: E731
                              for x in (s["k"], s["v"])]
    return _exact_rows(case, s, [(int(row[b]), int(n[b]), int(end[b])) for b in range(case["seqs"])], keys)
