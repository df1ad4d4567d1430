"""Measured cases of the 8-bit KV cache operators: the write (prompt and appended rows), the
read-back, the single-token decode attention over the cache, and SnapKV's selection writing its
kept rows into it.

The cache holds, per (layer, batch, KV head) unit, K and V in e4m3 codes with one power-of-two scale
for each block of 64 rows; the last n mod 64 rows, which do not fill a block, stay in bf16 (the tail).
A case is one of the operators at one size; run() is one pass through it, in its plain form (torch
operations in 32 bits) or, with own set, through the package's entry points.
"""

import math

import torch

own = False

BLOCK = 64      # rows of one scale
FP8 = torch.float8_e4m3fn


# ----------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------

def listed():
    return [
        # a padded batch of prompts of different lengths, one layer, 64-wide heads
        dict(name="write a ragged batch d64", op="write", layers=1, batch=16, kv_heads=12, dim=64,
             rows=1023, ragged=True),
        # long prompts over several layers at once
        dict(name="write 16k prompts", op="write", layers=8, batch=2, kv_heads=8, dim=128,
             rows=16384, ragged=False),
        # a few new tokens for every sequence of a batch, at ragged fill levels
        dict(name="append 5 tokens", op="append", layers=1, batch=16, kv_heads=8, dim=128,
             rows=5, filled=1100),
        # a chunk of a prompt appended to a long history
        dict(name="append a 700-token chunk", op="append", layers=4, batch=2, kv_heads=8, dim=128,
             rows=700, filled=5000),
        # one layer of a compact cache read back (to continue in bf16)
        dict(name="read a compact layer", op="read", layers=1, batch=2, kv_heads=8, dim=128,
             filled=1100),
        # a long cache read back
        dict(name="read a 30k cache", op="read", layers=4, batch=2, kv_heads=8, dim=128,
             filled=30001),
        # one layer's step of one short request: latency counts
        dict(name="decode one short request", op="decode", layers=1, batch=1, kv_heads=8, group=4,
             dim=128, filled=300, ragged=False),
        # the step over every layer's compact cache after SnapKV (budget 1024 and some decoded tokens)
        dict(name="decode compact caches", op="decode", layers=32, batch=2, kv_heads=8, group=4,
             dim=128, filled=1100, ragged=False),
        # a batch of requests of very different lengths, 64-wide heads, many heads to a KV head
        dict(name="decode a ragged batch d64", op="decode", layers=1, batch=48, kv_heads=4, group=8,
             dim=64, filled=8191, ragged=True),
        # the full cache of a long context, one head to a KV head
        dict(name="decode a 131k context", op="decode", layers=2, batch=1, kv_heads=32, group=1,
             dim=128, filled=131050, ragged=False),
        # SnapKV's selection on a short prompt: latency counts
        dict(name="keep 64 of 512", op="select", layers=1, batch=1, kv_heads=4, dim=64, rows=512,
             budget=64, window=8, pool=7),
        # SnapKV's selection over several layers' long prompts, its kept rows quantised as written
        dict(name="keep 1024 of 16k", op="select", layers=8, batch=2, kv_heads=8, dim=128,
             rows=16384, budget=1024, window=32, pool=7),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "append", "read", "decode", "decode", "select"])
    dim = rng.choice([64, 128, 128])
    c = dict(op=op, layers=rng.choice([1, 1, 2, 4]), batch=_log(rng, 1, 24),
             kv_heads=rng.choice([1, 2, 4, 8, 12, 32]), dim=dim)
    units = c["layers"] * c["batch"] * c["kv_heads"]
    most = max(64, min(131000, (1 << 22) // units))     # rows a unit, so that no case outgrows the listed ones
    if op == "write":
        c.update(rows=_log(rng, 1, min(most, 20000)), ragged=rng.random() < 0.5)
    elif op == "append":
        c.update(rows=_log(rng, 1, min(most, 1500)), filled=_log(rng, 1, min(most, 9000)))
    elif op == "read":
        c.update(filled=_log(rng, 1, min(most, 40000)))
    elif op == "decode":
        c.update(group=rng.choice([1, 2, 3, 4, 5, 7, 8]), filled=_log(rng, 1, most),
                 ragged=rng.random() < 0.5)
    else:
        c["rows"] = _log(rng, 200, max(400, min(most, 30000)))
        c["window"] = rng.choice([8, 16, 32])
        c["pool"] = rng.choice([1, 5, 7, 13])
        c["budget"] = rng.randint(c["window"] + 1, min(c["rows"] // 2, 2048))
    return c


# ----------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------

def _units(c):
    return (c["layers"], c["batch"], c["kv_heads"])


def _blocks_up(rows):
    return (rows + BLOCK - 1) // BLOCK * BLOCK


def _cap(c):
    """Rows a cache is allocated for: what it holds and what the call adds."""
    if c["op"] == "write":
        return _blocks_up(c["rows"])
    if c["op"] == "append":
        return _blocks_up(c["filled"] + c["rows"])
    if c["op"] == "read":
        return _blocks_up(c["filled"])
    if c["op"] == "decode":
        return _blocks_up(c["filled"] + 1)
    return _blocks_up(c["budget"] + BLOCK)


def _rows_like(units, rows, dim, gen):
    """K or V rows: normal values, some channels much larger than the rest, as keys have."""
    x = torch.randn(units + (rows, dim), generator=gen, device="cuda")
    boost = 1 + 7 * (torch.rand(units + (1, dim), generator=gen, device="cuda") < 0.05).float()
    return x.mul_(boost).to(torch.bfloat16)


def _lengths(c, most, gen):
    """Rows of each unit: the same for the heads and layers of a sequence."""
    Ly, B, H = _units(c)
    if c["op"] == "append" or c.get("ragged"):
        n = torch.randint(0, most + 1, (1, B, 1), generator=gen, device="cuda", dtype=torch.int32)
    else:
        n = torch.full((1, B, 1), most, device="cuda", dtype=torch.int32)
    return n.expand(Ly, B, H).contiguous()


def prepare(case, seed):
    """A dict of the inputs and of the cache's tensors, as a program holds them before the call."""
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    units, D, cap = _units(c), c["dim"], _cap(c)
    s = {"case": c}
    filled = c.get("filled", 0)
    cache = {
        "k_codes": torch.zeros(units + (cap, D), device="cuda", dtype=torch.uint8).view(FP8),
        "v_codes": torch.zeros(units + (cap, D), device="cuda", dtype=torch.uint8).view(FP8),
        "k_scale": torch.ones(units + (cap // BLOCK,), device="cuda"),
        "v_scale": torch.ones(units + (cap // BLOCK,), device="cuda"),
        "k_tail": torch.zeros(units + (BLOCK, D), device="cuda", dtype=torch.bfloat16),
        "v_tail": torch.zeros(units + (BLOCK, D), device="cuda", dtype=torch.bfloat16),
        "pos": torch.full(units + (cap,), -1, device="cuda", dtype=torch.int32),
        "n_valid": torch.zeros(units, device="cuda", dtype=torch.int32),
    }
    s["cache"] = cache
    if filled:
        n0 = _lengths(c, filled, gen)
        s["n0"] = n0
        for name in ("k", "v"):
            for layer in range(units[0]):    # a layer at a time: the bf16 rows are only passing through
                x = _rows_like((1,) + units[1:], cap, D, gen)
                codes, scale = _quantise(x.view(1, units[1], units[2], cap // BLOCK, BLOCK, D).float())
                cache[name + "_codes"][layer] = codes.view(units[1:] + (cap, D))
                cache[name + "_scale"][layer] = scale.view(units[1:] + (cap // BLOCK,))
                first = (n0[layer] // BLOCK * BLOCK).long()
                rows = (first.unsqueeze(-1) + torch.arange(BLOCK, device="cuda")).clamp(max=cap - 1)
                cache[name + "_tail"][layer] = torch.gather(
                    x[0], 2, rows.unsqueeze(-1).expand(units[1:] + (BLOCK, D)))
        at = torch.arange(cap, device="cuda", dtype=torch.int32)
        cache["pos"].copy_(torch.where(at < n0.unsqueeze(-1), at, -1))
        cache["n_valid"].copy_(n0)
    if c["op"] == "write":
        s["k"], s["v"] = (_rows_like(units, c["rows"], D, gen) for _ in "kv")
        s["lengths"] = _lengths(c, c["rows"], gen) if c["ragged"] else None
    elif c["op"] == "append":
        s["k"], s["v"] = (_rows_like(units, c["rows"], D, gen) for _ in "kv")
    elif c["op"] == "read":
        s["k_out"], s["v_out"] = (torch.zeros(units + (cap, D), device="cuda", dtype=torch.bfloat16)
                                  for _ in "kv")
    elif c["op"] == "decode":
        s["q"] = torch.randn((c["layers"], c["batch"], c["kv_heads"] * c["group"], D), generator=gen,
                             device="cuda").to(torch.bfloat16)
        s["k"], s["v"] = (_rows_like(units, 1, D, gen).squeeze(-2).contiguous() for _ in "kv")
    else:
        s["k"], s["v"] = (_rows_like(units, c["rows"], D, gen) for _ in "kv")
        # window votes: few positions hold most of the attention
        s["votes"] = torch.randn(units + (c["rows"],), generator=gen, device="cuda").mul_(2).exp_()
    return s


# ----------------------------------------------------------------------------------------------
# plain form
# ----------------------------------------------------------------------------------------------

def _quantise(x):
    """fp32 blocks [..., 64, D] -> e4m3 codes and the blocks' scales: the least power of two with
    max |x| <= 448 scale."""
    amax = x.abs().amax(dim=(-2, -1))
    mant, expo = torch.frexp(amax)                     # amax = mant 2^expo, 448 = 0.875 2^9
    e = torch.where(mant > 0.875, expo - 8, expo - 9)
    e = torch.where(amax > 0, e, 0).to(torch.int32)
    scale = ((e + 127) << 23).view(torch.float32)      # 2^e, exactly
    return (x / scale[..., None, None]).to(FP8), scale


def _put_rows(cache, name, x, start, count):
    """Writes rows x [..., m, D] at row start of each unit (count of them): whole blocks in codes,
    the rest in the tail.  Returns the new codes, scales and tail."""
    units, D = x.shape[:3], x.shape[-1]
    codes, scale, tail = (cache[name + t] for t in ("_codes", "_scale", "_tail"))
    cap, nb = codes.shape[3], codes.shape[3] // BLOCK
    start, count = start.long().unsqueeze(-1), count.long().unsqueeze(-1)
    first = start // BLOCK * BLOCK                     # the open block's first row
    end = start + count
    # the rows from the open block on: the tail's, then x's
    r = torch.arange(cap + BLOCK, device=x.device).expand(units + (cap + BLOCK,))
    from_x = (r >= start) & (r < end)
    wide = (r - start).clamp(0, x.shape[3] - 1).unsqueeze(-1).expand(-1, -1, -1, -1, D)
    rows = torch.gather(x, 3, wide)
    in_tail = (r >= first) & (r < start)
    back = (r - first).clamp(0, BLOCK - 1).unsqueeze(-1).expand(-1, -1, -1, -1, D)
    rows = torch.where(in_tail.unsqueeze(-1), torch.gather(tail, 3, back), rows)
    # whole blocks
    new_codes, new_scale = _quantise(rows[:, :, :, :cap].float().view(units + (nb, BLOCK, D)))
    b = torch.arange(nb, device=x.device) * BLOCK
    whole = (b >= first) & (b + BLOCK <= end)
    out_codes = torch.where(whole.repeat_interleave(BLOCK, -1).unsqueeze(-1),
                            new_codes.view(codes.shape).view(torch.uint8), codes.view(torch.uint8)).view(FP8)
    out_scale = torch.where(whole, new_scale, scale)
    # the open block after the write: its new rows; what is behind them stays
    last = end // BLOCK * BLOCK
    t = last + torch.arange(BLOCK, device=x.device)
    new_tail = torch.gather(rows, 3, t.unsqueeze(-1).expand(-1, -1, -1, -1, D))
    fresh = (t < end) & (t >= start)
    kept = (t < start) & (last == first)
    out_tail = torch.where((fresh | kept).unsqueeze(-1), new_tail, tail)
    return out_codes, out_scale, out_tail


def _put(s, start, count):
    cache, got = s["cache"], {}
    for name in ("k", "v"):
        got[name + "_codes"], got[name + "_scale"], got[name + "_tail"] = _put_rows(
            cache, name, s[name], start, count)
    return got


def _new_pos(cache, start, count, clear):
    at = torch.arange(cache["pos"].shape[-1], device="cuda", dtype=torch.int32)
    end = (start + count).unsqueeze(-1)
    return torch.where((at >= start.unsqueeze(-1)) & (at < end), at, -1 if clear else cache["pos"])


def _write(s):
    c, cache = s["case"], s["cache"]
    zero = torch.zeros(_units(c), device="cuda", dtype=torch.int32)
    n = s["lengths"] if s["lengths"] is not None else torch.full_like(zero, c["rows"])
    return {**_put(s, zero, n), "pos": _new_pos(cache, zero, n, True), "n_valid": n.clone()}


def _append(s):
    c, cache = s["case"], s["cache"]
    n0 = s["n0"]
    m = torch.full_like(n0, c["rows"])
    at = torch.arange(cache["pos"].shape[-1], device="cuda", dtype=torch.int32)
    new = (at >= n0.unsqueeze(-1)) & (at < (n0 + m).unsqueeze(-1))
    pos = torch.where(new, c["filled"] + at - n0.unsqueeze(-1), cache["pos"])
    return {**_put(s, n0, m), "pos": pos, "n_valid": n0 + m}


def _read(s):
    cache = s["cache"]
    units, cap, D = s["k_out"].shape[:3], s["k_out"].shape[3], s["k_out"].shape[4]
    n = s["n0"].long().unsqueeze(-1)
    first = n // BLOCK * BLOCK
    r = torch.arange(cap, device="cuda")
    got = {}
    for name in ("k", "v"):
        held = cache[name + "_codes"].float().view(units + (cap // BLOCK, BLOCK, D))
        held = (held * cache[name + "_scale"][..., None, None]).view(units + (cap, D))
        t = (r - first).clamp(0, BLOCK - 1).unsqueeze(-1).expand(-1, -1, -1, -1, D)
        tail = torch.gather(cache[name + "_tail"], 3, t).float()
        x = torch.where((r < first).unsqueeze(-1), held, tail).to(torch.bfloat16)
        got[name] = torch.where((r < n).unsqueeze(-1), x, s[name + "_out"])
    return got


def _decode(s):
    c, cache = s["case"], s["cache"]
    units, D, G = _units(c), c["dim"], c["group"]
    cap = cache["k_codes"].shape[3]
    n0 = s["n0"].long()
    first = (n0 // BLOCK * BLOCK).unsqueeze(-1)
    at = (n0 - n0 // BLOCK * BLOCK)[..., None, None].expand(units + (1, D))
    k_tail = cache["k_tail"].scatter(3, at, s["k"].unsqueeze(3))    # the step's token joins the tail
    v_tail = cache["v_tail"].scatter(3, at, s["v"].unsqueeze(3))
    live = torch.arange(BLOCK, device="cuda") <= (n0.unsqueeze(-1) - first)
    held = torch.arange(cap, device="cuda") < first

    q = s["q"].float().view(units + (G, D)) / math.sqrt(D)
    blocks = units + (cap // BLOCK, BLOCK, D)
    k = (cache["k_codes"].float().view(blocks) * cache["k_scale"][..., None, None]).view(units + (cap, D))
    s1 = torch.matmul(q, k.transpose(-1, -2)).masked_fill(~held.unsqueeze(3), -math.inf)
    s2 = torch.matmul(q, k_tail.float().transpose(-1, -2)).masked_fill(~live.unsqueeze(3), -math.inf)
    del k
    m = torch.maximum(s1.amax(-1, keepdim=True), s2.amax(-1, keepdim=True))
    p1, p2 = torch.exp(s1 - m), torch.exp(s2 - m)
    total = p1.sum(-1, keepdim=True) + p2.sum(-1, keepdim=True)
    v = (cache["v_codes"].float().view(blocks) * cache["v_scale"][..., None, None]).view(units + (cap, D))
    tail_v = torch.where(live.unsqueeze(-1), v_tail.float(), 0.0)
    o = (torch.matmul(p1, v) + torch.matmul(p2, tail_v)) / total
    del v
    # a block that the token filled is quantised after the step
    full = (n0 + 1) % BLOCK == 0
    b = torch.div(n0, BLOCK, rounding_mode="floor")
    got = {}
    for name, tail in (("k", k_tail), ("v", v_tail)):
        codes, scale = _quantise(tail.float())
        cc = cache[name + "_codes"].view(torch.uint8).view(blocks)
        to = b[..., None, None, None].expand(units + (1, BLOCK, D))
        cur = torch.gather(cc, 3, to)
        cc.scatter_(3, to, torch.where(full[..., None, None, None], codes.view(torch.uint8).unsqueeze(3), cur))
        sc = cache[name + "_scale"]
        cur = torch.gather(sc, 3, b.unsqueeze(-1))
        sc.scatter_(3, b.unsqueeze(-1), torch.where(full.unsqueeze(-1), scale.unsqueeze(-1), cur))
        tail = torch.where(full[..., None, None], cache[name + "_tail"], tail)   # its rows left the tail
        got[name + "_codes"], got[name + "_scale"], got[name + "_tail"] = cache[name + "_codes"], sc, tail
    r = torch.arange(cap, device="cuda")
    pos = torch.where(r == n0.unsqueeze(-1), c["filled"], cache["pos"])
    return {"out": o.to(torch.bfloat16).view(s["q"].shape), "pos": pos, "n_valid": s["n0"] + 1, **got}


def _select(s):
    c, cache = s["case"], s["cache"]
    units = _units(c)
    L, W, keep = c["rows"], c["window"], c["budget"] - c["window"]
    half = (c["pool"] - 1) // 2
    padded = torch.nn.functional.pad(s["votes"][..., :L - W], (half, half), value=-math.inf)
    pooled = padded.unfold(-1, c["pool"], 1).amax(-1)
    order = torch.sort(pooled, dim=-1, descending=True, stable=True).indices[..., :keep]
    pos = torch.cat([order.sort(-1).values,
                     torch.arange(L - W, L, device="cuda").expand(units + (W,))], -1)
    wide = pos.unsqueeze(-1).expand(-1, -1, -1, -1, c["dim"])
    rows = {"cache": cache, "k": torch.gather(s["k"], 3, wide), "v": torch.gather(s["v"], 3, wide)}
    n = torch.full(units, c["budget"], device="cuda", dtype=torch.int32)
    got = _put(rows, torch.zeros_like(n), n)
    all_pos = torch.full_like(cache["pos"], -1)
    all_pos[..., :c["budget"]] = pos.to(torch.int32)
    return {**got, "pos": all_pos, "n_valid": n}


# ----------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------


def _handle(s):
    """The package's cache over the state's tensors, which a program makes once and keeps."""
    if "handle" not in s:
        import attention_score_kv_snapkv_gb300 as kvc
        s["handle"] = (kvc, kvc.KV8Cache.from_tensors(**s["cache"]))
    return s["handle"]


def run(state):
    s, c = state, state["case"]
    cache = s["cache"]
    if c["op"] in ("append", "decode"):
        cache["n_valid"].copy_(s["n0"])        # every pass adds to the same fill level
    if not own:
        return {"write": _write, "append": _append, "read": _read, "decode": _decode,
                "select": _select}[c["op"]](s)
    kvc, handle = _handle(s)
    if c["op"] == "write":
        kvc.kv8_write(s["k"], s["v"], handle, lengths=s["lengths"])
    elif c["op"] == "append":
        kvc.kv8_append(s["k"], s["v"], handle, new_pos=c["filled"])
    elif c["op"] == "read":
        k, v = kvc.kv8_read(handle, k_out=s["k_out"], v_out=s["v_out"])
        return {"k": k, "v": v}
    elif c["op"] == "decode":
        out = kvc.kv8_decode_attn(s["q"], handle, k_new=s["k"], v_new=s["v"], new_pos=c["filled"])
        return {"out": out, **cache}
    else:
        kvc.snapkv_select_kv8(s["votes"], s["k"], s["v"], handle, keep_window=c["window"],
                              pool_kernel=c["pool"], budget=c["budget"])
    return dict(cache)


# ----------------------------------------------------------------------------------------------
# work and exact values
# ----------------------------------------------------------------------------------------------

def work(case):
    c = case
    u = c["layers"] * c["batch"] * c["kv_heads"]
    D = c["dim"]
    rows = c.get("rows", 0) * (0.5 if c.get("ragged") else 1.0)          # lengths are drawn evenly
    filled = c.get("filled", 0) * (0.5 if c.get("ragged") else 1.0)
    if c["op"] in ("write", "append"):
        return {"bytes": u * rows * D * 6.0 + u * rows * 4.0, "flops": 0}
    if c["op"] == "read":
        return {"bytes": u * filled * D * 6.0, "flops": 0}
    if c["op"] == "decode":
        held, tail = max(0.0, filled - 31.5), min(filled, 32.5)
        if not c.get("ragged"):
            held, tail = filled // BLOCK * BLOCK, filled % BLOCK
        return {"bytes": u * (held * D * 2.0 + (tail + 2) * D * 4.0 + held / BLOCK * 8.0
                              + c["group"] * D * 4.0),
                "flops": 4.0 * u * c["group"] * D * (filled + 1)}
    return {"bytes": u * (4.0 * c["rows"] + 6.0 * D * c["budget"] + 4.0 * c["budget"]), "flops": 0}


def _e4m3_positive():
    """The positive finite e4m3 values in order: 3 fraction bits, bias 7, least exponent -6."""
    got = []
    for code in range(1, 127):
        ex, fr = code >> 3, code & 7
        got.append(fr * 2.0 ** -9 if ex == 0 else (8 + fr) * 2.0 ** (ex - 10))
    return got


def _nearest(x):
    """x (64 bits, |x| <= 448) to the nearest e4m3 value, halves to the even code."""
    grid = torch.tensor([0.0] + _e4m3_positive(), device=x.device, dtype=torch.float64)
    a = x.abs()
    hi = torch.searchsorted(grid, a).clamp(1, grid.numel() - 1)       # grid[hi - 1] < a <= grid[hi]
    lo = hi - 1
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where(up < down, hi, torch.where(up > down, lo, torch.where(hi % 2 == 0, hi, lo)))
    return torch.copysign(grid[pick], x)


def _exact_blocks(x):
    """64-bit blocks [n, 64, D] -> their codes' values and scales."""
    top = x.abs().amax((1, 2))
    powers = torch.tensor([2.0 ** i for i in range(-126, 121)], device=x.device, dtype=torch.float64)
    scale = powers[torch.searchsorted(448.0 * powers, top)]            # the first with 448 scale >= top
    scale = torch.where(top > 0, scale, 1.0)
    return _nearest(x / scale[:, None, None]), scale


def _exact_unit(cache, u, name, old, fresh):
    """Codes, scales and tail of unit u of `name` after rows `fresh` (64 bits) follow its `old` rows."""
    codes = cache[name + "_codes"][u].double()
    scale = cache[name + "_scale"][u].double()
    tail = cache[name + "_tail"][u].double()
    first = old // BLOCK * BLOCK
    rows = torch.cat([tail[:old - first], fresh])
    n = rows.shape[0] // BLOCK
    if n:
        c, sc = _exact_blocks(rows[:n * BLOCK].view(n, BLOCK, -1))
        codes[first:first + n * BLOCK] = c.view(n * BLOCK, -1)
        scale[first // BLOCK:first // BLOCK + n] = sc
    rest = rows[n * BLOCK:]
    tail[:rest.shape[0]] = rest
    return codes, scale, tail


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    cache = s["cache"]
    Ly, B, H = _units(c)
    every = [(a, b, h) for a in range(Ly) for b in range(B) for h in range(H)]
    names = ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail")
    large = sum(cache[n].numel() for n in names) > 6e8       # then of the cache's outputs none
    if len(every) > 1024 or large and c["op"] != "decode":
        return None
    if c["op"] == "read":
        got = {}
        for name in ("k", "v"):
            out = s[name + "_out"].double()
            for u in every:
                n = int(s["n0"][u])
                first = n // BLOCK * BLOCK
                sc = cache[name + "_scale"][u][:first // BLOCK].double().repeat_interleave(BLOCK)
                out[u][:first] = cache[name + "_codes"][u][:first].double() * sc[:, None]
                out[u][first:n] = cache[name + "_tail"][u][:n - first].double()
            got[name] = out
        return got
    got = {n: None if large else torch.empty(cache[n].shape, device="cuda", dtype=torch.float64)
           for n in names}
    got["pos"], got["n_valid"] = None, None
    out = []
    for u in every:
        old = int(s["n0"][u]) if "n0" in s else 0
        fresh = {}
        if c["op"] == "select":
            W = c["window"]
            v = s["votes"][u][:c["rows"] - W].double()
            half = c["pool"] // 2
            top = torch.stack([torch.roll(torch.nn.functional.pad(v, (half, half), value=-1.0), -j)[:v.numel()]
                               for j in range(c["pool"])]).amax(0)
            # the largest first, equal ones in order of position
            order = torch.argsort(-top, stable=True)[:c["budget"] - W]
            rows = torch.cat([torch.sort(order).values, torch.arange(c["rows"] - W, c["rows"], device="cuda")])
            fresh = {n: s[n][u][rows].double() for n in ("k", "v")}
        elif c["op"] == "decode":
            fresh = {n: s[n][u][None].double() for n in ("k", "v")}
        else:
            n = c["rows"] if s.get("lengths") is None else int(s["lengths"][u])
            fresh = {k: s[k][u][:n].double() for k in ("k", "v")}
        if c["op"] == "decode":
            full = {}
            for name in ("k", "v"):
                first = old // BLOCK * BLOCK
                sc = cache[name + "_scale"][u][:first // BLOCK].double().repeat_interleave(BLOCK)
                full[name] = torch.cat([cache[name + "_codes"][u][:first].double() * sc[:, None],
                                        cache[name + "_tail"][u][:old - first].double(), fresh[name]])
            G = c["group"]
            q = s["q"][u[0], u[1], u[2] * G:(u[2] + 1) * G].double()
            w = torch.softmax(q @ full["k"].T / c["dim"] ** 0.5, dim=-1)
            out.append(w @ full["v"])
        for name in () if large else ("k", "v"):
            got[name + "_codes"][u], got[name + "_scale"][u], got[name + "_tail"][u] = _exact_unit(
                cache, u, name, old, fresh[name])
    if c["op"] == "decode":
        got["out"] = torch.stack(out).view(s["q"].shape)
    return got
