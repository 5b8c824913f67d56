"""Measured cases of the 4-bit paged cache and of what feeds it: appending to it,
attention over it, reading it back, the block tables and slot maps of a step,
and rotary positions of several axes.

`run` computes each operator in elementary torch operations, or, with `own`
set, through this library's entry points.  A case is a dict of plain values;
the ragged lengths of a case come from its own `len_seed`, the tensors from
the seed given to `prepare`.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GROUP = 32                   # channels that share a scale of the 4-bit cache
SEVENTH = 0.14285714924335479736328125     # 1 / 7 in 32 bits
K_SCALE_MOST = 9352.0        # 7 of it are within 16 bits


# ------------------------------------------------------------------ cases
def _axes(name, **kw):
    c = dict(op="axes", name=name, dtype="bf16", tokens=64, hq=32, hkv=8, dim=128,
             sections="16,24,24", interleaved=False, turns=False, own_freqs=False, fused=False,
             far=4096)
    c.update(kw)
    return c


def _axes_append(name, **kw):
    c = dict(op="axes_append", name=name, dtype="bf16", n=64, ones=0, q_lo=1, q_hi=1, ctx_lo=1024,
             ctx_hi=16384, hq=32, hkv=8, dim=128, page=16, layout="NHD", sections="16,24,24",
             interleaved=False, turns=False, own_freqs=False, far=4096, len_seed=31)
    c.update(kw)
    return c


def _step(name, **kw):
    c = dict(op="step", name=name, n=64, new_lo=1, new_hi=1, len_lo=1024, len_hi=16384, page=16,
             max_len=16448, requests=128, spare=64, len_seed=41)
    c.update(kw)
    return c


def _append(name, **kw):
    c = dict(op="append", name=name, dtype="bf16", n=64, ones=0, q_lo=1, q_hi=1, ctx_lo=1024,
             ctx_hi=16384, hkv=8, dim=128, page=16, layout="NHD", len_seed=51)
    c.update(kw)
    return c


def _gather(name, **kw):
    c = dict(op="gather", name=name, dtype="bf16", n=4, ones=0, q_lo=1024, q_hi=16384, ctx_lo=0,
             ctx_hi=0, hkv=8, dim=128, page=64, layout="NHD", len_seed=61)
    c.update(kw)
    return c


def _attn(name, **kw):
    c = dict(op="attn", name=name, dtype="bf16", n=1, ones=0, q_lo=1, q_hi=1, ctx_lo=1024,
             ctx_hi=16384, hq=32, hkv=8, dim=128, page=16, layout="NHD", window=0, sinks=0,
             len_seed=71)
    c.update(kw)
    return c


def listed():
    return [
        # q and k of a video's tokens, axes of their own frequencies, pairs side by side
        _axes("axes_video_32768", tokens=32768, hq=40, hkv=40, sections="16,24,24",
              interleaved=True, own_freqs=True, far=256),
        # a decoding step of a model that reads images: rotate q and k at their own
        # positions and store k and v for 64 sequences
        _axes_append("axes_append_decode_64"),
        # prompts with images in them, axes in turn along the frequencies
        _axes_append("axes_append_prompts", dtype="fp16", n=6, q_lo=500, q_hi=4000, ctx_lo=0,
                     ctx_hi=0, hq=16, hkv=4, sections="24,20,20", turns=True, page=64,
                     layout="HND", len_seed=32),
        # a decoding step of a full server: its tables, and the drafted token taken back
        _step("step_decode_64"),
        # prompts' chunks of a large batch: thousands of pages and tens of thousands of rows
        _step("step_prompts_256", n=256, new_lo=1, new_hi=400, len_lo=0, len_hi=8000, page=32,
              max_len=8448, requests=1024, spare=4096, len_seed=42),
        # one new token of each of 64 sequences into the 4-bit cache, and back
        _append("append_q4_decode_64"),
        # packed prompts of the varlen workload's shape into it, and back for the prompt's
        # own attention
        _append("append_q4_prompts", dtype="fp16", n=8, q_lo=1024, q_hi=16384, ctx_lo=0, ctx_hi=0,
                hkv=16, dim=80, page=64, layout="HND", len_seed=52),
        # a cached prefix of four sequences as 16-bit keys and values
        _gather("gather_prefixes"),
        # one sequence, one token, a short cache: latency
        _attn("decode_one_short_q4", ctx_lo=776, ctx_hi=776),
        # a decoding step of a full server: ragged lengths
        _attn("decode_64_q4", n=64),
        # checking five drafted tokens per sequence, sliding window and sinks
        _attn("draft5_window_q4", dtype="fp16", n=48, q_lo=5, q_hi=5, ctx_lo=64, ctx_hi=32768,
              hq=16, hkv=4, dim=64, page=32, window=1024, sinks=4, len_seed=73),
        # a chunk of a long prompt: 2048 new tokens over 63488 cached ones
        _attn("chunk_2048_of_65536_q4", q_lo=2048, q_hi=2048, ctx_lo=63488, ctx_hi=63488, page=64),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _unnamed(c):
    return {k: v for k, v in c.items() if k != "name"}


def draw(rng):
    dtype = rng.choice(["bf16", "fp16"])
    dim = rng.choice([128, 128, 64, 80, 96, 40, 8 * rng.randint(4, 16)])
    hkv = rng.choice([1, 2, 4, 8, 8, 16])
    hq = hkv * rng.choice([1, 2, 3, 4, 4, 5, 8])
    page = rng.choice([16, 16, 32, 64, 128, 256])
    layout = rng.choice(["NHD", "HND"])
    kind = rng.choice(["axes", "axes_append", "step", "append", "gather", "decode", "decode",
                       "chunk", "chunk", "mixed"])
    seed = rng.randint(1, 1 << 30)
    # axes: the head's pairs, or some of them, cut into two to four parts
    pairs = rng.choice([dim // 2, dim // 2, dim // 4, 8])
    cuts = sorted(rng.sample(range(1, pairs), rng.randint(1, min(3, pairs - 1))))
    parts = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
    turned = dict(sections=",".join(map(str, parts)), interleaved=rng.random() < 0.5,
                  turns=rng.random() < 0.4, own_freqs=rng.random() < 0.5,
                  far=_spread(rng, 100, 1 << 20))
    if kind == "axes":
        return _unnamed(_axes("", dtype=dtype, tokens=_spread(rng, 1, 32768), hq=hq, hkv=hkv,
                              dim=dim, fused=rng.random() < 0.5, **turned))
    if kind == "step":
        n = _spread(rng, 1, 512)
        new_hi = _spread(rng, 1, max(1, min(8192, 65536 // n)))
        len_hi = _spread(rng, 1, 32768)
        return _unnamed(_step("", n=n, new_lo=rng.choice([0, 1, new_hi]), new_hi=new_hi,
                              len_lo=rng.choice([0, len_hi // 2]), len_hi=len_hi, page=page,
                              max_len=len_hi + new_hi + rng.randint(0, 500),
                              requests=n + rng.choice([0, 5, 300]), spare=_spread(rng, 1, 8192),
                              len_seed=seed))
    if kind in ("append", "axes_append", "gather"):
        n = _spread(rng, 1, 128)
        top = max(1, min(16384, 60000 // n))
        rows = dict(dtype=dtype, n=n, ones=rng.choice([0, n // 2]), q_lo=1,
                    q_hi=_spread(rng, 1, top), ctx_lo=0, ctx_hi=rng.choice([0, 100, 5000]),
                    hkv=hkv, dim=dim, page=page, layout=layout, len_seed=seed)
        if kind == "axes_append":
            return _unnamed(_axes_append("", hq=hq, **rows, **turned))
        return _unnamed((_append if kind == "append" else _gather)("", **rows))
    window, sinks = rng.choice([(0, 0), (0, 0), (rng.randint(1, 4000), rng.randint(0, 40))])
    ones = 0
    if kind == "decode":
        n = _spread(rng, 1, 128)
        q_lo, q_hi = 1, rng.choice([1, 1, 1, 2, 4, 7])
        hi = _spread(rng, 16, min(65536, (1 << 20) // n))
    elif kind == "chunk":
        n = rng.choice([1, 1, 2, 3])
        q_hi = _spread(rng, 8, 4096 // n)
        q_lo = max(1, q_hi // 2)
        hi = _spread(rng, 16, 16384)
    else:
        n = rng.randint(3, 24)
        ones = rng.randint(1, n - 1)
        q_lo, q_hi = 2, _spread(rng, 8, 1000)
        hi = _spread(rng, 16, 8192)
    return _unnamed(_attn("", dtype=dtype, n=n, ones=ones, q_lo=q_lo, q_hi=q_hi,
                          ctx_lo=rng.choice([0, hi // 2]), ctx_hi=hi, hq=hq, hkv=hkv, dim=dim,
                          page=page, layout=layout, window=window, sinks=sinks, len_seed=seed))


def _lens(c):
    """Per sequence: new tokens and the cached length with them."""
    r = random.Random(c["len_seed"])
    q = [1 if s < c["ones"] else r.randint(c["q_lo"], c["q_hi"]) for s in range(c["n"])]
    ctx = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in q]
    return q, [a + b for a, b in zip(q, ctx)]


def _step_lens(c):
    r = random.Random(c["len_seed"])
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["n"])]
    return new, [r.randint(c["len_lo"], c["len_hi"]) for _ in new]


def _sections(c):
    return [int(x) for x in c["sections"].split(",")]


def _visible(first, last, window, sinks):
    """(row, key) pairs that rows at positions first..last see, and the keys that any of them sees."""
    if window <= 0:
        return (last * (last + 1) - first * (first - 1)) // 2 + (last - first + 1), last + 1
    pairs = sum(min(p + 1, min(sinks, max(0, p + 1 - window)) + min(window, p + 1))
                for p in range(first, last + 1))
    low = max(0, first - window + 1)
    return pairs, min(sinks, low) + last + 1 - low


def _cached(c):
    """Bytes of one key and value of every head in the 4-bit cache."""
    return c["hkv"] * 2 * (c["dim"] // 2 + 2 * -(-c["dim"] // GROUP))


def work(case):
    c = case
    if c["op"] == "step":
        new, old = _step_lens(c)
        pages = sum(-(-(a + b) // c["page"]) for a, b in zip(new, old))
        return {"bytes": 8 * pages + 16 * sum(new) + 24 * c["n"], "flops": 4.0 * sum(new)}
    if c["op"] == "axes":
        rows, turned, axes = c["tokens"] * (c["hq"] + c["hkv"]), 2 * sum(_sections(c)), len(_sections(c))
        return {"bytes": rows * c["dim"] * 4 + c["tokens"] * 8 * axes + turned * 4,
                "flops": rows * turned * 3}
    q, kv = _lens(c)
    tokens = sum(q)
    row = tokens * c["hkv"] * c["dim"]
    if c["op"] == "axes_append":
        turned = tokens * (c["hq"] + c["hkv"]) * 2 * sum(_sections(c))
        return {"bytes": row * 8 + tokens * c["hq"] * c["dim"] * 4 + tokens * 8 * len(_sections(c)),
                "flops": turned * 3}
    if c["op"] == "append":
        return {"bytes": row * 8 + tokens * _cached(c), "flops": row * 8}
    if c["op"] == "gather":
        return {"bytes": row * 4 + tokens * _cached(c), "flops": row * 4}
    pairs = keys = 0
    for a, b in zip(q, kv):
        p, k = _visible(b - a, b - 1, c["window"], c["sinks"])
        pairs, keys = pairs + p, keys + k
    return {"bytes": tokens * c["hq"] * c["dim"] * 4 + keys * _cached(c),
            "flops": 4.0 * pairs * c["hq"] * c["dim"]}


# ----------------------------------------------------------------- inputs
def _turns(c, dev):
    """Each pair's axis, and its frequency in 64 bits."""
    parts = _sections(c)
    half = sum(parts)
    if c["turns"]:           # axis 0, 1, 2, 0, 1, 2, ... while an axis has pairs left
        left, order = list(parts), []
        while len(order) < half:
            order += [a for a in range(len(parts)) if left[a] > 0]
            left = [max(0, x - 1) for x in left]
    else:
        order = [a for a, x in enumerate(parts) for _ in range(x)]
    axes = torch.tensor(order, dtype=torch.uint8, device=dev)
    at, span = torch.arange(half, dtype=torch.float64, device=dev), float(half)
    if c["own_freqs"]:       # every axis from the highest frequency on
        seen, place = [0] * len(parts), []
        for a in order:
            place.append(seen[a] / parts[a])
            seen[a] += 1
        at, span = torch.tensor(place, dtype=torch.float64, device=dev), 1.0
    return axes, 10000.0 ** (-at / span)


def _grid(c, tokens, g, dev):
    """Positions (axes, tokens): text, where all axes advance together, with
    images and video in between, whose axes count frames, rows and columns."""
    axes = len(_sections(c))
    t = torch.arange(tokens, device=dev)
    start = int(torch.randint(0, max(1, c["far"] - 64), (1,), generator=g, device=dev))
    wide = 8 + int(torch.randint(0, 57, (1,), generator=g, device=dev))
    spans = (wide * wide, wide, 1)
    image = (t // 97) % 3 != 0
    rows = [t // 7 + torch.where(image, (t // spans[min(a, 2)]) % wide, t % 7) for a in range(axes)]
    return (torch.stack(rows) + start).clamp_(max=c["far"] - 1).contiguous()


def _codes(x, most):
    """Four-bit codes of x (..., channels), a multiple of 32, packed, and their scales."""
    top = x.unflatten(-1, (-1, GROUP)).abs().amax(-1)
    scale = (top * SEVENTH).clamp(max=most).half()
    wide = scale.float().repeat_interleave(GROUP, -1)
    inv = torch.where(wide > 0, torch.ones_like(wide) / wide, 0.0)
    n = (torch.round(x * inv).clamp(-7, 7) + 8).to(torch.uint8)
    return n[..., 0::2] | n[..., 1::2] << 4, scale


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    s = {"case": c}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    if c["op"] == "step":
        new, old = _step_lens(c)
        n, page = c["n"], c["page"]
        width = -(-c["max_len"] // page)
        have = [-(-x // page) for x in old]
        total = sum(have) + c["spare"]
        order = torch.randperm(total, generator=g, device=dev).int()
        req = torch.randperm(c["requests"], generator=g, device=dev)[:n].int()
        s["req"], s["new"] = req, torch.tensor(new, dtype=torch.int32, device=dev)
        s["keep"] = torch.tensor(old, dtype=torch.int32, device=dev)
        s["lens"] = torch.zeros(c["requests"], dtype=torch.int32, device=dev)
        s["lens"][req.long()] = s["keep"]
        s["table"] = torch.full((c["requests"], width), -1, dtype=torch.int32, device=dev)
        used = torch.tensor(have, device=dev)
        row = torch.repeat_interleave(torch.arange(n, device=dev), used)
        slot = torch.arange(sum(have), device=dev) - (used.cumsum(0) - used)[row]
        s["table"][req.long()[row], slot] = order[:sum(have)]
        s["free"] = torch.full((total,), -1, dtype=torch.int32, device=dev)
        s["free"][:c["spare"]] = order[sum(have):]
        s["left"] = torch.tensor([c["spare"]], dtype=torch.int32, device=dev)
        s["rows"], s["max_q"] = sum(new), max(new)
        return s

    dt = TYPES[c["dtype"]]
    if c["op"] == "axes":
        t, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["dim"]
        if c["fused"]:
            qkv = normal(t, hq + 2 * hkv, d).to(dt)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        else:
            s["q"], s["k"] = normal(t, hq, d).to(dt), normal(t, hkv, d).to(dt)
        s["pos"] = _grid(c, t, g, dev)
        s["axes"], s["inv_freq"] = _turns(c, dev)
        return s

    q_len, kv_len = _lens(c)
    n, page, hkv, d = c["n"], c["page"], c["hkv"], c["dim"]
    tokens = sum(q_len)
    width = max(-(-x // page) for x in kv_len)
    used = [-(-x // page) for x in kv_len]
    pool = sum(used) + 3
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(n, width, dtype=torch.int32, device=dev)
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = order[at:at + u]
        at += u
    starts = [0]
    for x in q_len:
        starts.append(starts[-1] + x)
    s["block"] = table
    s["cu_q"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    s["kv_lens"] = torch.tensor(kv_len, dtype=torch.int32, device=dev)
    s["max_q"], s["max_kv"], s["rows"] = max(q_len), max(kv_len), tokens
    nhd = c["layout"] == "NHD"
    if c["op"] == "axes_append":
        shape = (pool, page, hkv, d) if nhd else (pool, hkv, page, d)
        s["k"], s["v"] = normal(*shape).to(dt), normal(*shape).to(dt)
        s["k_new"], s["v_new"] = normal(tokens, hkv, d).to(dt), normal(tokens, hkv, d).to(dt)
        s["q"] = normal(tokens, c["hq"], d).to(dt)
        s["pos"] = _grid(c, tokens, g, dev)
        s["axes"], s["inv_freq"] = _turns(c, dev)
        return s
    groups, dp = -(-d // GROUP), 64 if d <= 64 else 128
    shape = (pool, page, hkv, GROUP * groups) if nhd else (pool, hkv, page, GROUP * groups)
    mean = normal(hkv, d) * 3.0              # a fixed per-channel offset of K
    s["k_mean"] = torch.zeros(hkv, dp, device=dev)
    s["k_mean"][:, :d] = mean
    s["v_scale"] = torch.zeros(hkv, dp, device=dev)
    s["v_scale"][:, :d] = (4.0 + torch.rand(hkv, d, generator=g, device=dev)) / 448.0
    for name, most in (("k", K_SCALE_MOST), ("v", 1.0)):
        x = normal(*shape)
        x[..., d:] = 0.0
        s[name], scale = _codes(x if name == "k" else x * 1.4, most)
        s[name + "_groups"] = torch.zeros(pool, hkv, page, dp // GROUP, dtype=torch.float16, device=dev)
        s[name + "_groups"][..., :groups] = scale.transpose(1, 2) if nhd else scale
    if c["op"] == "append":
        s["k_new"] = (normal(tokens, hkv, d) + mean).to(dt)
        s["v_new"] = normal(tokens, hkv, d).to(dt)
    elif c["op"] == "attn":
        s["q"] = normal(tokens, c["hq"], d).to(dt)
    return s


# ------------------------------------------------------------ plain forms
def _turn(x, pos, axes, inv_freq, interleaved):
    """x [T, H, D] rotated in 32 bits; the angles of far positions need 64."""
    a = (pos[axes.long()].T.double() * inv_freq)[:, None]
    cos, sin = a.cos().float(), a.sin().float()
    r = 2 * inv_freq.numel()
    x = x.float()
    if interleaved:
        x1, x2 = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1).flatten(-2)
    else:
        x1, x2 = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1)
    return torch.cat((y, x[..., r:]), -1)


def _plain_axes(s):
    f = s["pos"], s["axes"], s["inv_freq"], s["case"]["interleaved"]
    return _turn(s["q"], *f).to(s["q"].dtype), _turn(s["k"], *f).to(s["k"].dtype)


def _places(s):
    """Each new token's sequence and position."""
    t = torch.arange(s["rows"], device=s["cu_q"].device)
    seq = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    return seq, s["kv_lens"].long()[seq] - s["cu_q"].long()[seq + 1] + t


def _slots(s):
    seq, pos = _places(s)
    page = s["case"]["page"]
    return s["block"].long()[seq, pos // page], pos % page


def _plain_axes_append(s):
    c = s["case"]
    page, slot = _slots(s)
    f = s["pos"], s["axes"], s["inv_freq"], c["interleaved"]
    at = (lambda x: x) if c["layout"] == "NHD" else (lambda x: x.transpose(1, 2))
    at(s["k"])[page, slot] = _turn(s["k_new"], *f).to(s["k"].dtype)
    at(s["v"])[page, slot] = s["v_new"]
    return {"k": s["k"], "v": s["v"], "q": _turn(s["q"], *f).to(s["q"].dtype)}


def _plain_step(s):
    """The tables of the step; then every new token is taken back."""
    c = s["case"]
    page, req = c["page"], s["req"].long()
    old, new = s["lens"][req].long(), s["new"].long()
    n, width = old.numel(), s["table"].shape[1]
    have, after = (old + page - 1) // page, (old + new + page - 1) // page
    need = after - have
    upto = need.cumsum(0)
    free = s["left"][0].long()
    fits = ((need == 0) | (upto <= free)) & (old + new <= c["max_len"])
    got = torch.where(fits, need, 0)
    end = torch.where(fits, have + need, have)
    # the pages: those of the request, then from the stack's end
    j = torch.arange(width, device=req.device)
    from_stack = free - 1 - (upto - need)[:, None] - (j - have[:, None])
    fresh = s["free"].long()[from_stack.clamp(0, s["free"].numel() - 1)]
    table = torch.where(j < have[:, None], s["table"][req].long(), fresh)
    table = torch.where(j < end[:, None], table, -1)
    cu = torch.cat((torch.zeros_like(new[:1]), new.cumsum(0)))
    seq = torch.repeat_interleave(torch.arange(n, device=req.device), new, output_size=s["rows"])
    pos = old[seq] + torch.arange(s["rows"], device=req.device) - cu[seq]
    pos = torch.where(fits[seq], pos, -1)
    slots = torch.where(pos >= 0, table[seq, pos.clamp(min=0) // page] * page + pos % page, -1)
    kv_lens = torch.where(fits, old + new, 0)
    s["table"][req] = torch.where(j < end[:, None], table.int(), s["table"][req])
    s["lens"][req] = torch.where(fits, old + new, old).int()
    s["left"] -= got.sum().int()
    # back to the lengths from before: the pages go onto the stack in the order that
    # undoes the step
    now, keep = s["lens"][req].long(), s["keep"].long()
    back = (now + page - 1) // page - (keep + page - 1) // page
    first = (back.cumsum(0) - back)[:, None] - ((keep + page - 1) // page)[:, None]
    total = s["left"][0].long() + back.sum()
    gone = (j >= ((keep + page - 1) // page)[:, None]) & (j < ((now + page - 1) // page)[:, None])
    to = torch.where(gone, total - 1 - first - j, s["free"].numel())
    room = torch.cat((s["free"], s["free"][:1]))
    room[to] = s["table"][req]
    s["free"].copy_(room[:-1])
    s["lens"][req] = torch.minimum(now, keep).int()
    s["left"] += back.sum().int()
    return {"cu_q": cu.int(), "kv_lens": kv_lens.int(), "block_table": table.int(),
            "positions": pos, "slots": slots, "denied": (~fits).sum().int(), "lens": s["lens"],
            "free": s["free"], "left": s["left"]}


def _values(s, name, packed, groups):
    """What packed codes (..., rows of bytes) with their groups' scales stand for, in 32 bits."""
    d = s["case"]["dim"]
    n = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)[..., :d].float() - 8.0
    x = n * groups.float().repeat_interleave(GROUP, -1)[..., :d]
    return x if name == "k" else x * (64.0 * s["v_scale"][:, :d])


def _plain_gather(s):
    """The rows' keys and values as 16 bits."""
    c = s["case"]
    page, slot = _slots(s)
    at = (lambda x: x) if c["layout"] == "NHD" else (lambda x: x.transpose(1, 2))
    k, v = (_values(s, n, at(s[n])[page, slot], s[n + "_groups"].transpose(1, 2)[page, slot])
            for n in ("k", "v"))
    return (k + s["k_mean"][:, :c["dim"]]).to(TYPES[c["dtype"]]), v.to(TYPES[c["dtype"]])


def _plain_append(s):
    c = s["case"]
    d = c["dim"]
    page, slot = _slots(s)
    inv = torch.where(s["v_scale"] > 0, torch.ones_like(s["v_scale"]) / (64.0 * s["v_scale"]), 0.0)
    x = torch.stack((s["k_new"].float() - s["k_mean"][:, :d], s["v_new"].float() * inv[:, :d]))
    x = torch.nn.functional.pad(x, (0, -d % GROUP))
    k, k_groups = _codes(x[0], K_SCALE_MOST)
    v, v_groups = _codes(x[1], 1.0)
    at = (lambda x: x) if c["layout"] == "NHD" else (lambda x: x.transpose(1, 2))
    at(s["k"])[page, slot], at(s["v"])[page, slot] = k, v
    s["k_groups"].transpose(1, 2)[page, slot, :, :k_groups.shape[-1]] = k_groups
    s["v_groups"].transpose(1, 2)[page, slot, :, :v_groups.shape[-1]] = v_groups
    return _plain_gather(s)


def _plain_attn(s):
    c = s["case"]
    dev = s["q"].device
    hq, hkv, d, page = c["hq"], c["hkv"], c["dim"], c["page"]
    j = torch.arange(s["max_kv"], device=dev)
    pages, slots = s["block"].long()[:, j // page], (j % page).expand(c["n"], -1)
    at = (lambda x: x) if c["layout"] == "NHD" else (lambda x: x.transpose(1, 2))
    k, v = (_values(s, n, at(s[n])[pages, slots], s[n + "_groups"].transpose(1, 2)[pages, slots])
            for n in ("k", "v"))
    seq, pos = _places(s)
    row = torch.arange(seq.numel(), device=dev) - s["cu_q"].long()[seq]
    q = torch.zeros(c["n"], s["max_q"], hq, d, device=dev)
    q[seq, row] = s["q"].float()
    p = torch.full((c["n"], s["max_q"]), -1, dtype=torch.int64, device=dev)
    p[seq, row] = pos
    # [n, kv head, group * rows, keys]
    q = q.view(c["n"], s["max_q"], hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(d))
    seen = j <= p[..., None]
    if c["window"] > 0:
        seen = seen & ((j > p[..., None] - c["window"]) | (j < c["sinks"]))
    x = x.view(c["n"], hkv, hq // hkv, s["max_q"], s["max_kv"])
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == float("-inf"), 0.0, m)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.flatten(2, 3), v.permute(0, 2, 1, 3)).view(c["n"], hkv, hq // hkv, s["max_q"], d)
    o = o / torch.where(total == 0, 1.0, total)
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3)[seq, row].to(s["q"].dtype)


# ------------------------------------------------- the library's own calls
def _own_cache(sage, s):
    if "cache" not in s:    # kept by a serving program for the life of its cache
        c = s["case"]
        more = {} if "k_groups" not in s else dict(k_groups=s["k_groups"], v_groups=s["v_groups"],
                                                   k_mean=s["k_mean"], v_scale=s["v_scale"],
                                                   head_dim=c["dim"])
        s["cache"] = sage.PagedCache(s["k"], s["v"], c["layout"], **more)
        s["batch"] = sage.PagedBatch(s["cu_q"], s["kv_lens"], s["block"], s["max_q"], s["max_kv"])
        s["ws"] = sage.alloc_workspace_paged()
    return s["cache"], s["batch"], s["ws"]


def _own_axes(s):
    from quantized_attention_smooth_gb300 import sage
    return sage.rope(s["q"], s["k"], s["pos"], s["inv_freq"], interleaved=s["case"]["interleaved"],
                     axes=s["axes"])


def _own_axes_append(s):
    from quantized_attention_smooth_gb300 import sage
    cache, batch, ws = _own_cache(sage, s)
    q = sage.kv_append(cache, batch, s["k_new"], s["v_new"], q=s["q"], inv_freq=s["inv_freq"],
                       interleaved=s["case"]["interleaved"], positions=s["pos"], axes=s["axes"],
                       ws=ws)
    return {"k": s["k"], "v": s["v"], "q": q}


def _own_step(s):
    from quantized_attention_smooth_gb300 import sage
    c = s["case"]
    if "pool" not in s:
        s["pool"] = sage.PagePool(s["free"], s["left"], s["table"], s["lens"], c["page"])
        s["plan"] = sage.PagedPlan(s["pool"], c["n"], s["rows"], s["max_q"], c["max_len"])
        s["ws"] = sage.alloc_workspace_paged()
    pool, plan = s["pool"], s["plan"]
    sage.paged_step(pool, plan, s["req"], s["new"], ws=s["ws"])
    sage.paged_trim(pool, s["req"], s["keep"], ws=s["ws"])
    return {"cu_q": plan.cu_q, "kv_lens": plan.kv_lens, "block_table": plan.block_table,
            "positions": plan.positions, "slots": plan.slots, "denied": plan.denied,
            "lens": s["lens"], "free": s["free"], "left": s["left"]}


def _own_append(s):
    from quantized_attention_smooth_gb300 import sage
    cache, batch, ws = _own_cache(sage, s)
    sage.kv_append(cache, batch, s["k_new"], s["v_new"], ws=ws)
    return sage.kv_gather(cache, batch, s["rows"], TYPES[s["case"]["dtype"]], ws=ws)


def _own_gather(s):
    from quantized_attention_smooth_gb300 import sage
    cache, batch, ws = _own_cache(sage, s)
    return sage.kv_gather(cache, batch, s["rows"], TYPES[s["case"]["dtype"]], ws=ws)


def _own_attn(s):
    from quantized_attention_smooth_gb300 import sage
    cache, batch, ws = _own_cache(sage, s)
    return sage.attn_paged(cache, batch, s["q"], window=s["case"]["window"],
                           sinks=s["case"]["sinks"], ws=ws)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"axes": _own_axes, "axes_append": _own_axes_append, "step": _own_step,
                "append": _own_append, "gather": _own_gather, "attn": _own_attn}[op](state)
    return {"axes": _plain_axes, "axes_append": _plain_axes_append, "step": _plain_step,
            "append": _plain_append, "gather": _plain_gather, "attn": _plain_attn}[op](state)


# ------------------------------------------------------------- definition
def _exact_turn(x, s):
    """Each pair as a complex number times its axis' unit number, in 64 bits."""
    x = x.double().clone()
    f, pos = s["inv_freq"], s["pos"].double()
    half = f.numel()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if s["case"]["interleaved"] else (
        slice(0, half), slice(half, 2 * half))
    angle = torch.stack([pos[int(axis)] * f[i] for i, axis in enumerate(s["axes"].tolist())], -1)
    z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    x[..., a], x[..., b] = z.real, z.imag
    return x


def _exact_codes(x, most):
    """x (T, heads, d) after four-bit quantisation, in 64 bits but for the scale's own 16."""
    d = x.shape[-1]
    out = torch.zeros_like(x)
    for a in range(0, d, GROUP):
        part = x[..., a:a + GROUP]
        scale = (part.abs().amax(-1, keepdim=True) / 7).clamp(max=most).half().double()
        code = torch.where(scale > 0, part / torch.where(scale > 0, scale, 1.0), 0.0)
        out[..., a:a + GROUP] = code.round().clamp(-7, 7) * scale
    return out


def _exact_rows(s, i, b, h=None):
    """Keys (less their mean) and values of sequence i, positions 0 .. b - 1, in 64 bits."""
    c = s["case"]
    d, page = c["dim"], c["page"]
    pages = s["block"][i, :-(-b // page)].long()
    heads = range(c["hkv"]) if h is None else [h]
    out = []
    for name in ("k", "v"):
        rows = []
        for head in heads:
            packed = s[name][pages, :, head] if c["layout"] == "NHD" else s[name][pages, head]
            packed = packed.reshape(-1, packed.shape[-1])[:b]
            x = torch.empty(packed.shape[0], 2 * packed.shape[1], dtype=torch.float64,
                            device=packed.device)
            x[:, 0::2], x[:, 1::2] = (packed % 16).double() - 8, (packed // 16).double() - 8
            scale = s[name + "_groups"][pages, head].reshape(-1, s[name + "_groups"].shape[-1])[:b]
            for g in range(0, d, GROUP):
                x[:, g:g + GROUP] *= scale[:, g // GROUP, None].double()
            x = x[:, :d]
            rows.append(x if name == "k" else x * 64 * s["v_scale"][head, :d].double())
        out.append(torch.stack(rows, 1))
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "step":    # whole numbers
        return None
    if c["op"] == "axes":
        return _exact_turn(s["q"], s), _exact_turn(s["k"], s)
    q_len, kv_len = _lens(c)
    d, hkv, page = c["dim"], c["hkv"], c["page"]
    start = 0
    if c["op"] == "axes_append":
        turned, k, v = _exact_turn(s["k_new"], s), s["k"].double(), s["v"].double()
        for i, (a, b) in enumerate(zip(q_len, kv_len)):
            pos = torch.arange(b - a, b, device=k.device)
            pg, sl = s["block"][i].long()[pos // page], pos % page
            rows = slice(start, start + a)
            if c["layout"] == "NHD":
                k[pg, sl], v[pg, sl] = turned[rows], s["v_new"][rows].double()
            else:
                k[pg, :, sl], v[pg, :, sl] = turned[rows], s["v_new"][rows].double()
            start += a
        return {"k": k, "v": v, "q": _exact_turn(s["q"], s)}
    if c["op"] == "append":
        mean, unit = s["k_mean"][:, :d].double(), 64 * s["v_scale"][:, :d].double()
        return (_exact_codes(s["k_new"].double() - mean, K_SCALE_MOST) + mean,
                _exact_codes(s["v_new"].double() / unit, 1.0) * unit)
    if c["op"] == "gather":
        rows = [[x[b - a:] for x in _exact_rows(s, i, b)]
                for i, (a, b) in enumerate(zip(q_len, kv_len))]
        return (torch.cat([r[0] for r in rows]) + s["k_mean"][:, :d].double(),
                torch.cat([r[1] for r in rows]))
    if work(c)["flops"] > 5e12:
        return None
    group = c["hq"] // hkv
    out = torch.zeros(sum(q_len), c["hq"], d, dtype=torch.float64, device=s["q"].device)
    for i, (a, b) in enumerate(zip(q_len, kv_len)):
        pos = torch.arange(b - a, b, device=out.device)[:, None]
        key = torch.arange(b, device=out.device)[None]
        hidden = key > pos
        if c["window"] > 0:
            hidden |= (key <= pos - c["window"]) & (key >= c["sinks"])
        for h in range(hkv):
            kh, vh = (x[:, 0] for x in _exact_rows(s, i, b, h))
            for r in range(group):
                x = s["q"][start:start + a, h * group + r].double() @ kh.T * (d ** -0.5)
                x = torch.softmax(x.masked_fill_(hidden, float("-inf")), -1)
                out[start:start + a, h * group + r] = x @ vh
        start += a
    return out
