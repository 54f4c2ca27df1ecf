"""Cases of the key/value cache operators: rotary positions with several axes,
blocks and slots for new rows, appending rows to a cache held in 8 bits, and
attention over that cache.

Every case runs in two forms on the same inputs: the operator's plain form
(elementary torch operations in 32 bits, or 64 where an angle needs them) and
the library's entry points. The cache is kept in blocks of tokens, each block
(block_tokens, d) bytes of e4m3 per head with one fp32 scale for keys and one
for values; a block table maps a sequence's blocks to the cache's.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one generated token per sequence: its q and k get their positions
        dict(name="rotary_step", op="rotary", B=16, T=1, h=8, h_kv=8, d=128, sections="16,24,24",
             per_axis=False, interleaved=False, inverse=False, far=1000000, dtype="bf16"),
        # a video prompt: time, height and width of every patch, q and k of all heads
        dict(name="rotary_video", op="rotary", B=2, T=8192, h=16, h_kv=16, d=128,
             sections="16,24,24", per_axis=False, interleaved=False, inverse=False, far=40000,
             dtype="bf16"),
        # gradients of q and k of an image's patches (rows, columns), fp32, odd length
        dict(name="rotary_image_grad", op="rotary", B=4, T=1023, h=12, h_kv=12, d=64,
             sections="16,16", per_axis=True, interleaved=True, inverse=True, far=64,
             dtype="f32"),
        # a generation step of many sequences: a few of them cross into a new block
        dict(name="reserve_step", op="reserve", B=64, n=1, block_tokens=64, lo=1, hi=8192,
             short=False),
        # ragged prompts and follow-up turns, more of them than the free blocks can take
        dict(name="reserve_prompts", op="reserve", B=48, n=8192, block_tokens=16, lo=0, hi=20000,
             short=True),
        # one generated token per sequence goes into its partly filled block
        dict(name="append_step", op="append", B=16, n=1, h_kv=8, d_h=128, d_vh=128,
             block_tokens=64, lo=4096, hi=8192, dtype="bf16"),
        # whole prompts go into fresh and partly filled blocks
        dict(name="append_prompt", op="append", B=2, n=8192, h_kv=16, d_h=128, d_vh=128,
             block_tokens=64, lo=0, hi=100, dtype="bf16"),
        # short ragged turns, unequal head sizes, small blocks, fp32
        dict(name="append_ragged", op="append", B=5, n=77, h_kv=3, d_h=80, d_vh=48,
             block_tokens=16, lo=3, hi=200, dtype="f32"),
        # the start of a few conversations: two rows each, fp32 queries
        dict(name="attention_short", op="attention", B=3, n_q=2, h=12, h_kv=12, d_h=64, d_vh=64,
             block_tokens=16, lo=5, hi=1000, dtype="f32"),
        # a generation step over long caches, a key/value head for each query head
        dict(name="attention_step", op="attention", B=16, n_q=1, h=8, h_kv=8, d_h=128, d_vh=128,
             block_tokens=64, lo=4096, hi=8192, dtype="bf16"),
        # four drafted tokens to verify, four query heads to a key/value head, many long caches
        dict(name="attention_drafted", op="attention", B=32, n_q=4, h=32, h_kv=8, d_h=128,
             d_vh=128, block_tokens=32, lo=100, hi=32768, dtype="bf16"),
        # a piece of a prompt after what is cached of it
        dict(name="attention_piece", op="attention", B=2, n_q=512, h=16, h_kv=4, d_h=128,
             d_vh=128, block_tokens=64, lo=6000, hi=8192, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """An integer spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("rotary", "reserve", "append", "attention", "attention"))
    if op == "rotary":
        d = rng.choice((32, 64, 80, 96, 128, 256))
        axes = rng.choice((1, 2, 3))
        pairs = d // 2 if rng.random() < 0.7 else d // 4
        cuts = sorted(rng.sample(range(1, pairs), axes - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
        h = rng.choice((1, 4, 8, 12, 16, 32))
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, T=_log(rng, 1, max(1, min(9000, (1 << 26) // (B * h * d)))), h=h,
                    h_kv=max(1, h // rng.choice((1, 2, 4))), d=d,
                    sections=",".join(map(str, sections)), per_axis=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.3,
                    far=_log(rng, 64, 2000000), dtype=rng.choice(("bf16", "bf16", "f32")))
    bt = rng.choice((16, 32, 64, 128))
    if op == "reserve":
        lo = rng.choice((0, _log(rng, 1, 2000)))
        return dict(op=op, B=_log(rng, 1, 256), n=_log(rng, 1, 9000), block_tokens=bt, lo=lo,
                    hi=lo + _log(rng, 1, 20000), short=rng.random() < 0.3)
    d_h = rng.choice((32, 64, 80, 96, 128, 128, 256))
    d_vh = d_h if rng.random() < 0.7 else rng.choice((32, 48, 64, 128, 256))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    h_kv = rng.choice((1, 2, 4, 8, 12))
    B = _log(rng, 1, 64)
    if op == "append":
        lo = rng.choice((0, _log(rng, 1, 3000)))
        return dict(op=op, B=B, n=_log(rng, 1, max(1, min(9000, (1 << 25) // (B * h_kv * 256)))),
                    h_kv=h_kv, d_h=d_h, d_vh=d_vh, block_tokens=bt, lo=lo,
                    hi=lo + _log(rng, 1, 3000), dtype=dtype)
    n_q = rng.choice((1, 1, 2, _log(rng, 1, 300)))
    hi = _log(rng, 16, max(64, min(60000, (1 << 21) // (B * h_kv))))
    lo = rng.randint(1, hi)
    h = h_kv * rng.choice((1, 2, 4, 8))
    n_q = max(1, min(n_q, (1 << 26) // (B * h * (hi + n_q))))
    return dict(op=op, B=B, n_q=n_q, h=h, h_kv=h_kv, d_h=d_h, d_vh=d_vh, block_tokens=bt, lo=lo,
                hi=hi, dtype=dtype)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _spread(B, lo, hi, turn):
    """B integers over [lo, hi], both ends among them, the same for every seed."""
    v = [lo + round((hi - lo) * ((b * 0.6180339887498949 + turn) % 1.0)) for b in range(B)]
    v[0] = hi
    if B > 1:
        v[-1] = lo
    return v


def _lengths(case):
    """Per sequence: positions in the cache before the new rows, and new rows."""
    B = case["B"]
    if case["op"] == "attention":
        new = _spread(B, max(1, case["n_q"] // 2), case["n_q"], 0.3) if case["n_q"] > 8 else \
            [case["n_q"]] * B
        return [max(0, t - m) for t, m in zip(_spread(B, case["lo"], case["hi"], 0.0), new)], new
    new = _spread(B, max(1, case["n"] // 3), case["n"], 0.3)
    return _spread(B, case["lo"], case["hi"], 0.0), new


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pow2_scale(amax):
    """The smallest power of two s with amax / s <= 448 (at least 2^-126)."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-126, 127)
    e = torch.where(amax > 0, e, -126)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _filled(n_blocks, h, bt, d, g):
    """A cache of normal values: bytes of e4m3, and the scale of each block and head."""
    codes = torch.empty((n_blocks, h, bt, d), dtype=torch.uint8, device="cuda")
    scale = torch.empty((n_blocks, h), device="cuda")
    step = max(1, (1 << 27) // (h * bt * d))
    for i in range(0, n_blocks, step):
        x = torch.randn((min(step, n_blocks - i), h, bt, d), device="cuda", generator=g)
        s = _pow2_scale(x.abs().amax(dim=(2, 3)))
        scale[i:i + step] = s
        codes[i:i + step] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scale


def _table(total, bt, n_blocks, max_blocks, g):
    """Blocks of every sequence, scattered over the cache; -1 where there is none yet."""
    need = [-(-t // bt) for t in total]
    ids = torch.randperm(n_blocks, device="cuda", generator=g)[:sum(need)].to(torch.int32)
    table = torch.full((len(total), max_blocks), -1, dtype=torch.int32, device="cuda")
    rows = torch.repeat_interleave(torch.arange(len(need)), torch.tensor(need))
    cols = torch.cat([torch.arange(k) for k in need])
    table[rows.cuda(), cols.cuda()] = ids
    return table


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "rotary":
        dt = DTYPES[case["dtype"]]
        B, T, d = case["B"], case["T"], case["d"]
        s["sections"] = [int(x) for x in case["sections"].split(",")]
        s["Q"] = torch.randn((B, case["h"], T, d), device="cuda", generator=g).to(dt)
        s["K"] = torch.randn((B, case["h_kv"], T, d), device="cuda", generator=g).to(dt)
        s["positions"] = torch.randint(0, case["far"], (len(s["sections"]), B, T),
                                       device="cuda", generator=g, dtype=torch.int32)
        # a user's program keeps the frequencies, in the form that its call takes
        s["frequencies"] = torch.tensor(_frequencies(s["sections"], case["per_axis"]),
                                        dtype=torch.float64, device="cuda")
        s["axis"] = torch.repeat_interleave(
            torch.arange(len(s["sections"])), torch.tensor(s["sections"])).cuda()
        if own:
            from head_scaled_dot_gb300 import mha
            s["steps"] = mha.rotary_steps(s["sections"], per_axis=case["per_axis"])
            s["out"] = (torch.empty_like(s["Q"]), torch.empty_like(s["K"]))
        return s
    cached, new = _lengths(case)
    bt = case["block_tokens"]
    total = [a + b for a, b in zip(cached, new)]
    max_blocks = -(-max(total) // bt) + 1
    used = sum(-(-t // bt) for t in total)
    n_blocks = used + max(2, used // 16)
    s["cached_len"], s["new_len"], s["total_len"] = _ints(cached), _ints(new), _ints(total)
    if case["op"] == "reserve":
        held = sum(-(-t // bt) for t in cached)
        order = torch.randperm(n_blocks, device="cuda", generator=g).to(torch.int32)
        table = torch.full((case["B"], max_blocks), -1, dtype=torch.int32, device="cuda")
        need = torch.tensor([-(-t // bt) for t in cached])
        rows = torch.repeat_interleave(torch.arange(case["B"]), need)
        cols = torch.cat([torch.arange(int(k)) for k in need])
        table[rows.cuda(), cols.cuda()] = order[:held]
        s["block_table"] = table
        free = (n_blocks - held) * 2 // 3 if case["short"] else n_blocks - held
        s["free_blocks"] = order[held:].contiguous()
        s["n_free"] = _ints([free])
        if own:
            s["out"] = (torch.empty(case["B"], dtype=torch.int32, device="cuda"),
                        torch.empty((case["B"], case["n"]), dtype=torch.int64, device="cuda"),
                        torch.empty(1, dtype=torch.int32, device="cuda"))
        return s
    dt = DTYPES[case["dtype"]]
    h_kv, d_h, d_vh = case["h_kv"], case["d_h"], case["d_vh"]
    s["block_table"] = _table(total, bt, n_blocks, max_blocks, g)
    s["K_cache"], s["K_scale"] = _filled(n_blocks, h_kv, bt, d_h, g)
    s["V_cache"], s["V_scale"] = _filled(n_blocks, h_kv, bt, d_vh, g)
    if case["op"] == "append":
        B, n = case["B"], case["n"]
        s["K"] = torch.randn((B, h_kv, n, d_h), device="cuda", generator=g).to(dt)
        # values of a few tokens stand out, as they do in earnest
        loud = 1 + 7 * (torch.rand((B, 1, n, 1), device="cuda", generator=g) < 0.05)
        s["V"] = (torch.randn((B, h_kv, n, d_vh), device="cuda", generator=g) * loud).to(dt)
        i = torch.arange(n, device="cuda")[None]
        pos = s["cached_len"][:, None] + i
        block = torch.gather(s["block_table"], 1, (pos // bt).clamp(max=max_blocks - 1).long())
        s["slot_map"] = torch.where(i < s["new_len"][:, None], block.long() * bt + pos % bt, -1)
        return s
    s["Q"] = torch.randn((case["B"], case["h"], case["n_q"], d_h), device="cuda",
                         generator=g).to(dt)
    s["c"] = d_h ** -0.5
    if own:
        from head_scaled_dot_gb300 import mha
        s["out"] = torch.empty((case["B"], case["n_q"], case["h"] * d_vh), dtype=dt,
                               device="cuda")
        s["workspace"] = torch.empty(
            mha.attention_cache_workspace_size(case["B"], case["n_q"], case["h"], h_kv, d_h,
                                               d_vh), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _frequencies(sections, per_axis, base=10000.0):
    if per_axis:
        return [base ** (-j / m) for m in sections for j in range(m)]
    return [base ** (-j / sum(sections)) for j in range(sum(sections))]


def _rotate(x, cos, sin, interleaved):
    """Each pair (a, b) of a row becomes (a cos - b sin, a sin + b cos)."""
    half = cos.shape[-1]
    f, rest = x[..., :2 * half].float(), x[..., 2 * half:]
    if interleaved:
        a, b = f[..., 0::2], f[..., 1::2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = f[..., :half], f[..., half:]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((y.to(x.dtype), rest), dim=-1)


def _plain_rotary(s):
    pos = s["positions"][s["axis"]].double()                 # (pairs, B, T)
    angle = (pos * s["frequencies"][:, None, None]).permute(1, 2, 0)[:, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if s["inverse"]:
        sin = -sin
    return {"Q": _rotate(s["Q"], cos, sin, s["interleaved"]),
            "K": _rotate(s["K"], cos, sin, s["interleaved"])}


def _plain_reserve(s):
    bt, n = s["block_tokens"], s["n"]
    have = (s["cached_len"] + (bt - 1)) // bt
    need = (s["cached_len"] + s["new_len"] + (bt - 1)) // bt - have
    last = torch.cumsum(need, 0, dtype=torch.int32)
    fits = (need == 0) | (last <= s["n_free"])
    got = torch.where(fits, need, 0)
    used = torch.where(fits, last, 0).amax()
    table = s["block_table"]
    col = torch.arange(table.shape[1], device="cuda", dtype=torch.int32)[None]
    fresh = (col >= have[:, None]) & (col < (have + got)[:, None])
    taken = (s["n_free"] - 1 - (last - need)[:, None] - (col - have[:, None]))
    ids = s["free_blocks"][taken.clamp(0, s["free_blocks"].numel() - 1).long()]
    table.copy_(torch.where(fresh, ids, table))
    new = torch.where(fits, s["new_len"], 0)
    i = torch.arange(n, device="cuda", dtype=torch.int32)[None]
    pos = s["cached_len"][:, None] + i
    block = torch.gather(table, 1, (pos // bt).clamp(max=table.shape[1] - 1).long())
    slot = torch.where(i < new[:, None], block.long() * bt + pos % bt, -1)
    return {"block_table": table, "total_len": s["cached_len"] + new, "slot_map": slot,
            "n_free": s["n_free"] - used}


def _quantise(x, scale):
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _plain_append_one(x, slots, codes, scales, bt):
    """Rows x (B, h, n, d) into their blocks. A block's scale is the smallest
    power of two that its rows fit, and never falls while it holds rows: where
    new rows raise it, the rows already there are rounded to it anew."""
    B, h, n, d = x.shape
    first = slots[:, 0] % bt                                  # offset of an item's first row
    count = (slots >= 0).sum(1)
    last_part = (first + count - 1) // bt
    part = torch.arange(n // bt + 2, device="cuda")[None].minimum(last_part[:, None])
    off = torch.arange(bt, device="cuda")[None, None]
    row = part[:, :, None] * bt - first[:, None, None] + off  # (B, parts, bt)
    fresh = (row >= 0) & (row < count[:, None, None])
    kept = row < 0
    at = row.clamp(0, n - 1)
    some = (part * bt - first[:, None]).clamp(min=0)
    block = torch.gather(slots, 1, some) // bt                # (B, parts)
    new = x.float().permute(0, 2, 1, 3)[torch.arange(B, device="cuda")[:, None, None], at]
    new = torch.where(fresh[..., None, None], new, 0)         # (B, parts, bt, h, d)
    need = _pow2_scale(new.abs().amax(dim=(2, 4)))            # (B, parts, h)
    before = scales[block]
    scale = torch.where(kept.any(2)[..., None], torch.maximum(before, need), need)
    there = codes[block]                                      # (B, parts, h, bt, d)
    again = _quantise(there.view(torch.float8_e4m3fn).float() * before[..., None, None],
                      scale[..., None, None])
    again = torch.where((scale > before)[..., None, None], again.view(torch.uint8), there)
    put = _quantise(new.permute(0, 1, 3, 2, 4), scale[..., None, None]).view(torch.uint8)
    out = torch.where(fresh[:, :, None, :, None], put, there)
    out = torch.where(kept[:, :, None, :, None], again, out)
    codes[block] = out
    scales[block] = scale


def _plain_append(s):
    bt = s["block_tokens"]
    _plain_append_one(s["K"], s["slot_map"], s["K_cache"], s["K_scale"], bt)
    _plain_append_one(s["V"], s["slot_map"], s["V_cache"], s["V_scale"], bt)
    return _cache_of(s)


def _cache_of(s):
    return {"K_cache": s["K_cache"].view(torch.float8_e4m3fn), "K_scale": s["K_scale"],
            "V_cache": s["V_cache"].view(torch.float8_e4m3fn), "V_scale": s["V_scale"]}


def _gathered(codes, scales, table):
    """The rows of every sequence (B, h, blocks * block_tokens, d), in fp32."""
    ids = table.clamp(min=0).long()
    x = codes[ids].view(torch.float8_e4m3fn).float() * scales[ids][..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attention(s):
    Q = s["Q"]
    B, h, n_q, d_h = Q.shape
    h_kv = s["h_kv"]
    K = _gathered(s["K_cache"], s["K_scale"], s["block_table"])
    V = _gathered(s["V_cache"], s["V_scale"], s["block_table"])
    total, new = s["total_len"][:, None, None, None], s["new_len"][:, None, None, None]
    key = torch.arange(K.shape[2], device="cuda")[None, None, None]
    i = torch.arange(n_q, device="cuda")[None, None, :, None]
    sees = ((key <= total - new + i) & (i < new))             # (B, 1, n_q, keys)
    V = torch.where(key.transpose(2, 3) < total, V, 0)
    q = Q.float().reshape(B, h_kv, h // h_kv * n_q, d_h)
    scores = (q @ K.transpose(2, 3)).view(B, h, n_q, -1) * s["c"]
    scores = scores.masked_fill(~sees, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -math.inf, top, 0))
    p = (p / p.sum(-1, keepdim=True).clamp(min=1e-30)).view(B, h_kv, h // h_kv * n_q, -1)
    z = (p @ V).view(B, h, n_q, -1).transpose(1, 2)
    return {"Z": z.flatten(2, 3).to(Q.dtype)}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _library(s):
    from head_scaled_dot_gb300 import mha
    if s["op"] == "rotary":
        Q, K = mha.rotary(s["Q"], s["K"], s["positions"], s["steps"], s["sections"],
                          interleaved=s["interleaved"], inverse=s["inverse"], out=s["out"])
        return {"Q": Q, "K": K}
    if s["op"] == "reserve":
        total, slots, n_free = mha.cache_reserve(
            s["cached_len"], s["new_len"], s["free_blocks"], s["n_free"], s["block_table"],
            s["block_tokens"], s["n"], out=s["out"])
        return {"block_table": s["block_table"], "total_len": total, "slot_map": slots,
                "n_free": n_free}
    if s["op"] == "append":
        mha.cache_append(s["K"], s["V"], s["slot_map"], s["K_cache"], s["V_cache"], s["K_scale"],
                         s["V_scale"])
        return _cache_of(s)
    return {"Z": mha.attention_cache(s["Q"], s["K_cache"], s["V_cache"], s["K_scale"],
                                     s["V_scale"], s["block_table"], s["total_len"], s["c"],
                                     new_len=s["new_len"], causal_tail=True, out=s["out"],
                                     workspace=s["workspace"])}


def run(state):
    if own:
        return _library(state)
    return {"rotary": _plain_rotary, "reserve": _plain_reserve, "append": _plain_append,
            "attention": _plain_attention}[state["op"]](state)


def work(case):
    if case["op"] == "rotary":
        rows, es = case["B"] * case["T"], 2 if case["dtype"] == "bf16" else 4
        values = rows * (case["h"] + case["h_kv"]) * case["d"]
        axes = case["sections"].count(",") + 1
        pairs = sum(int(x) for x in case["sections"].split(","))
        return {"bytes": 2 * values * es + 4 * axes * rows,
                "flops": 6 * rows * (case["h"] + case["h_kv"]) * pairs}
    cached, new = _lengths(case)
    bt, B = case["block_tokens"], case["B"]
    if case["op"] == "reserve":
        fresh = sum(-(-(a + m) // bt) + (-a // bt) for a, m in zip(cached, new))
        return {"bytes": 12 * B + 8 + 8 * fresh + 8 * B * case["n"], "flops": B * case["n"]}
    es = 2 if case["dtype"] == "bf16" else 4
    width = case["h_kv"] * (case["d_h"] + case["d_vh"])
    if case["op"] == "append":
        parts = sum(-(-(a % bt + m) // bt) for a, m in zip(cached, new))
        return {"bytes": sum(new) * (width * (es + 1) + 8) + 8 * case["h_kv"] * parts,
                "flops": 3 * sum(new) * width}
    total = sum(a + m for a, m in zip(cached, new))
    seen = sum(m * a + m * (m + 1) // 2 for a, m in zip(cached, new))
    blocks = sum(-(-(a + m) // bt) for a, m in zip(cached, new))
    ends = case["h"] * (case["d_h"] + case["d_vh"]) * es
    return {"bytes": total * width + blocks * (4 + 8 * case["h_kv"]) + sum(new) * ends + 8 * B,
            "flops": 2 * seen * case["h"] * (case["d_h"] + case["d_vh"])}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _e4m3(x):
    """x rounded to the nearest e4m3 value, ties to even, in float64."""
    e = torch.frexp(x.abs())[1].sub(1).clamp(min=-6)
    ulp = ((e - 3).long() + 1023 << 52).view(torch.float64)
    return (torch.round(x / ulp) * ulp).clamp(-E4M3_MAX, E4M3_MAX)


_BYTE_VALUES = []


def _byte_values():
    """The 256 values of e4m3 by byte: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    if not _BYTE_VALUES:
        for c in range(256):
            e, m = c >> 3 & 15, c & 7
            v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
            _BYTE_VALUES.append(-v if c & 128 else v)
    return torch.tensor(_BYTE_VALUES, dtype=torch.float64, device="cuda")


def _exact_rotary(s):
    out = {}
    w = [f / (2 * math.pi) for f in s["frequencies"].tolist()]
    turn = torch.tensor(w, dtype=torch.float64, device="cuda")
    p = s["positions"][s["axis"]].permute(1, 2, 0).double()
    whole = p * s["frequencies"]
    whole = whole - 2 * math.pi * torch.floor(p * turn)
    rot = torch.polar(torch.ones_like(whole), -whole if s["inverse"] else whole)[:, None]
    m = rot.shape[-1]
    for name in ("Q", "K"):
        x = s[name].double()
        y = x.clone()
        ia = torch.arange(m, device="cuda") * (2 if s["interleaved"] else 1)
        ib = ia + (1 if s["interleaved"] else m)
        z = torch.complex(x[..., ia], x[..., ib]) * rot
        y[..., ia], y[..., ib] = z.real, z.imag
        out[name] = y
    return out


def _exact_append(s):
    bt, vals = s["block_tokens"], _byte_values()
    out = {}
    for name in ("K", "V"):
        x, codes = s[name].double(), s[name + "_cache"]
        cache = vals[codes.long()]
        scale = s[name + "_scale"].double().clone()
        slots = s["slot_map"].cpu()
        for b in range(x.shape[0]):
            mine = slots[b][slots[b] >= 0]
            i = 0
            while i < len(mine):
                block, o = int(mine[i]) // bt, int(mine[i]) % bt
                m = min(bt - o, len(mine) - i)
                rows = x[b, :, i:i + m]
                amax = rows.abs().amax(dim=(1, 2))
                half, e = torch.frexp(amax / E4M3_MAX)
                e = torch.where(half == 0.5, e - 1, e).clamp(min=-126)
                need = (e.long() + 1023 << 52).view(torch.float64)
                new = torch.maximum(scale[block], need) if o else need
                if o:
                    ratio = (scale[block] / new)[:, None, None]
                    cache[block, :, :o] = _e4m3(cache[block, :, :o] * ratio)
                cache[block, :, o:o + m] = _e4m3(rows / new[:, None, None])
                scale[block] = new
                i += m
        out[name + "_cache"], out[name + "_scale"] = cache, scale
    return out


def _exact_attention(s):
    B, h, n_q, d_h = s["Q"].shape
    h_kv, bt, vals = s["h_kv"], s["block_tokens"], _byte_values()
    total, new = s["total_len"].tolist(), s["new_len"].tolist()
    Z = torch.zeros((B, n_q, h, s["d_vh"]), dtype=torch.float64, device="cuda")
    for b in range(B):
        ids = s["block_table"][b, :-(-total[b] // bt)].long()

        def rows(codes, scale):
            x = vals[codes[ids].long()] * scale[ids].double()[:, :, None, None]
            return x.transpose(0, 1).flatten(1, 2)[:, :total[b]]

        K, V = rows(s["K_cache"], s["K_scale"]), rows(s["V_cache"], s["V_scale"])
        limit = total[b] - new[b] + torch.arange(new[b], device="cuda")
        hides = torch.arange(total[b], device="cuda")[None] > limit[:, None]
        for j in range(h):
            a = s["Q"][b, j, :new[b]].double() @ K[j * h_kv // h].T * s["c"]
            a[hides] = -math.inf
            Z[b, :new[b], j] = torch.softmax(a, -1) @ V[j * h_kv // h]
    return {"Z": Z.flatten(2, 3)}


def exact(case, seed):
    if case["op"] == "reserve":
        return None
    return {"rotary": _exact_rotary, "append": _exact_append,
            "attention": _exact_attention}[case["op"]](prepare(case, seed))
