"""The paged-cache operators' measured cases: rotary positions, appending to a
paged cache and attention of new tokens over it.

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


# ------------------------------------------------------------------ cases
def _rope(name, **kw):
    c = dict(op="rope", name=name, dtype="bf16", tokens=64, hq=32, hkv=8, dim=128, rotary=128,
             interleaved=False, scaling="none", fused=False, far=131072)
    c.update(kw)
    return c


def _append(name, **kw):
    c = dict(op="append", name=name, dtype="bf16", n=64, ones=0, q_lo=1, q_hi=1, ctx_lo=1024,
             ctx_hi=16384, hq=32, hkv=8, dim=128, page=16, layout="NHD", q8=False, rotary=128,
             interleaved=False, scaling="none", len_seed=11)
    c.update(kw)
    return c


def _attn(name, **kw):
    c = dict(op="attn", name=name, dtype="bf16", n=1, ones=0, q_lo=1, q_hi=1, ctx_lo=1024,
             ctx_hi=16384, hq=32, hkv=8, dim=128, page=16, layout="NHD", q8=False, window=0,
             sinks=0, len_seed=21)
    c.update(kw)
    return c


def listed():
    return [
        # one decoding step of 64 sequences, far positions: launch latency
        _rope("rope_decode_64", scaling="yarn"),
        # a packed prefill's q and k, views into one fused projection, half of the head rotated
        _rope("rope_prefill_fused", dtype="fp16", tokens=16000, hq=40, hkv=40, rotary=64,
              interleaved=True, scaling="linear", fused=True, far=32768),
        # one decoding step: rotate q and k and store k and v for 64 sequences
        _append("append_decode_64", scaling="yarn"),
        # packed prompts of the varlen workload's shape into the quantised cache
        _append("append_q8_prefill", dtype="fp16", n=8, q_lo=1024, q_hi=16384, ctx_lo=0, ctx_hi=0,
                hq=16, hkv=16, dim=80, page=64, layout="HND", q8=True, rotary=0, len_seed=12),
        # one sequence, one token, a short cache: latency
        _attn("decode_one_short", ctx_lo=776, ctx_hi=776),
        # a decoding step of a full server: ragged lengths, 16-bit cache
        _attn("decode_64", n=64),
        # the same over the quantised cache
        _attn("decode_64_q8", n=64, q8=True, page=64, layout="HND", len_seed=22),
        # checking five drafted tokens per sequence, sliding window and sinks
        _attn("draft5_window", dtype="fp16", n=48, q_lo=5, q_hi=5, ctx_lo=64, ctx_hi=32768, hq=16,
              hkv=4, dim=64, page=32, window=1024, sinks=4, len_seed=23),
        # a chunk of a long prompt: 2048 new tokens over 30720 cached ones
        _attn("chunk_2048_of_32768", q_lo=2048, q_hi=2048, ctx_lo=30720, ctx_hi=30720, page=64),
        # chunked prefill with decoding sequences in one batch, every head its own keys
        _attn("mixed_d80", dtype="fp16", n=20, ones=16, q_lo=200, q_hi=1500, ctx_lo=100,
              ctx_hi=12000, hq=16, hkv=16, dim=80, page=32, layout="HND", len_seed=24),
        # chunks over the quantised cache
        _attn("chunks_q8", n=3, q_lo=700, q_hi=1400, ctx_lo=2000, ctx_hi=14000, page=128, q8=True,
              len_seed=25),
        # whole prompts: the causal GQA prefill's shape, two sequences
        _attn("prefill_2x8192", n=2, q_lo=8192, q_hi=8192, ctx_lo=0, ctx_hi=0, page=128,
              layout="HND"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "fp16"])
    dim = rng.choice([128, 128, 64, 80, 96, 40, 8 * rng.randint(4, 16)])
    hkv = rng.choice([1, 2, 4, 8, 8, 16])
    hq = hkv * rng.choice([1, 2, 3, 4, 4, 5, 8])
    page = rng.choice([16, 16, 32, 64, 128, 256])
    layout = rng.choice(["NHD", "HND"])
    kind = rng.choice(["rope", "append", "append_q8", "decode", "decode", "chunk", "chunk", "mixed"])
    if kind == "rope":
        tokens = _spread(rng, 1, 16000)
        rotary = rng.choice([dim, dim // 2 // 8 * 8, 16])
        return {k: v for k, v in _rope(
            "", dtype=dtype, tokens=tokens, hq=hq, hkv=hkv, dim=dim, rotary=rotary,
            interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "yarn"]),
            fused=rng.random() < 0.5, far=_spread(rng, 100, 1 << 20)).items() if k != "name"}
    seed = rng.randint(1, 1 << 30)
    if kind.startswith("append"):
        q8 = kind == "append_q8"
        n = _spread(rng, 1, 128)
        top = max(1, min(16384, 60000 // n))
        return {k: v for k, v in _append(
            "", dtype=dtype, n=n, ones=rng.choice([0, n // 2]), q_lo=1, q_hi=_spread(rng, 1, top),
            ctx_lo=0, ctx_hi=rng.choice([0, 100, 5000]), hq=hq, hkv=hkv, dim=dim, page=page,
            layout=layout, q8=q8, rotary=0 if q8 else rng.choice([0, dim, 16]),
            interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "yarn"]),
            len_seed=seed).items() if k != "name"}
    window, sinks = rng.choice([(0, 0), (0, 0), (rng.randint(1, 4000), rng.randint(0, 40))])
    q8 = rng.random() < 0.4
    if kind == "decode":
        n = _spread(rng, 1, 128)
        q_hi = rng.choice([1, 1, 1, 2, 4, 7])
        ones, q_lo = 0, 1
        hi = _spread(rng, 16, min(65536, (1 << 20) // n))
    elif kind == "chunk":
        n, ones = rng.choice([1, 1, 2, 3]), 0
        q_hi = _spread(rng, 8, 4096 // n)
        q_lo = max(1, q_hi // 2)
        hi = _spread(rng, 16, 16384)
    else:
        n = rng.randint(3, 24)
        ones = rng.randint(1, n - 1)
        q_lo, q_hi = 2, _spread(rng, 8, 1000)
        hi = _spread(rng, 16, 8192)
    return {k: v for k, v in _attn(
        "", dtype=dtype, n=n, ones=ones, q_lo=q_lo, q_hi=q_hi, ctx_lo=rng.choice([0, hi // 2]),
        ctx_hi=hi, hq=hq, hkv=hkv, dim=dim, page=page, layout=layout, q8=q8, window=window,
        sinks=sinks, len_seed=seed).items() if k != "name"}


def _lens(c):
    """Per sequence: new tokens and the cached length with them."""
    r = random.Random(c["len_seed"])
    q = [1 if s < c["ones"] else r.randint(c["q_lo"], c["q_hi"]) for s in range(c["n"])]
    ctx = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in q]
    return q, [a + b for a, b in zip(q, ctx)]


def _visible(first, last, window, sinks):
    """(row, key) pairs that rows at positions first..last see, and the keys that any of them sees."""
    if window <= 0:
        return (last * (last + 1) - first * (first - 1)) // 2 + (last - first + 1), last + 1
    pairs = sum(min(p + 1, min(sinks, max(0, p + 1 - window)) + min(window, p + 1))
                for p in range(first, last + 1))
    low = max(0, first - window + 1)
    return pairs, min(sinks, low) + last + 1 - low


def work(case):
    c = case
    if c["op"] == "rope":
        rows = c["tokens"] * (c["hq"] + c["hkv"])
        return {"bytes": rows * c["dim"] * 4 + c["tokens"] * 8 + c["rotary"] * 4,
                "flops": rows * c["rotary"] * 3}
    q, kv = _lens(c)
    tokens = sum(q)
    if c["op"] == "append":
        row = tokens * c["hkv"] * c["dim"]
        out = row * 2 + tokens * c["hkv"] * 4 if c["q8"] else row * 4
        turned = tokens * (c["hq"] + c["hkv"]) * c["rotary"]
        return {"bytes": row * 4 + out + (tokens * c["hq"] * c["dim"] * 4 if c["rotary"] else 0),
                "flops": turned * 3 + row * 4}
    pairs = keys = 0
    for a, b in zip(q, kv):
        p, k = _visible(b - a, b - 1, c["window"], c["sinks"])
        pairs, keys = pairs + p, keys + k
    per_key = c["hkv"] * (c["dim"] * 2 + 4) if c["q8"] else c["hkv"] * c["dim"] * 4
    return {"bytes": tokens * c["hq"] * c["dim"] * 4 + keys * per_key,
            "flops": 4.0 * pairs * c["hq"] * c["dim"]}


# ----------------------------------------------------------------- inputs
def _frequencies(c, dev):
    """inv_freq [rotary / 2] in 64 bits and the factor on cos and sin."""
    half = c["rotary"] // 2
    f = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
    if c["scaling"] == "linear":
        return f / 4.0, 1.0
    if c["scaling"] == "yarn":    # long wavelengths are stretched by 8, short ones kept, a ramp between
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return f * (keep + (1 - keep) / 8.0), 0.1 * math.log(8.0) + 1.0
    return f, 1.0


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    dt = TYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    s = {"case": c}
    if c["op"] == "rope":
        t, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["dim"]
        if c["fused"]:
            qkv = normal(t, hq + 2 * hkv, d)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        else:
            s["q"], s["k"] = normal(t, hq, d), normal(t, hkv, d)
        s["pos"] = torch.randint(0, c["far"], (t,), generator=g, device=dev)
        s["inv_freq"], s["mscale"] = _frequencies(c, dev)
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
    s["table"] = table
    s["cu_q"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    s["kv_lens"] = torch.tensor(kv_len, dtype=torch.int32, device=dev)
    s["max_q"], s["max_kv"] = max(q_len), max(kv_len)
    shape = (pool, page, hkv, d) if c["layout"] == "NHD" else (pool, hkv, page, d)
    if c["q8"]:
        mean = torch.randn(hkv, d, generator=g, device=dev) * 3.0    # a fixed per-channel offset of K
        dp = 64 if d <= 64 else 128
        s["k_mean"] = torch.zeros(hkv, dp, device=dev)
        s["k_mean"][:, :d] = mean
        s["v_scale"] = torch.zeros(hkv, dp, device=dev)
        s["v_scale"][:, :d] = (4.0 + torch.rand(hkv, d, generator=g, device=dev)) / 448.0
        by_head = (lambda m: m[:, :d]) if c["layout"] == "NHD" else (lambda m: m[:, None, :d])
        x = torch.randn(*shape, generator=g, device=dev)
        top = x.abs().amax(-1, keepdim=True)
        s["k"] = torch.round(x * (127.0 / top)).to(torch.int8)
        scale = (top / 127.0).squeeze(-1)
        s["k_scale"] = (scale.transpose(1, 2) if c["layout"] == "NHD" else scale).contiguous()
        x = torch.randn(*shape, generator=g, device=dev)
        s["v"] = (x / by_head(s["v_scale"])).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        s["k"], s["v"] = normal(*shape), normal(*shape)
    if c["op"] == "append":
        if c["q8"]:
            s["k_new"] = (torch.randn(tokens, hkv, d, generator=g, device=dev) + mean).to(dt)
        else:
            s["k_new"] = normal(tokens, hkv, d)
        s["v_new"] = normal(tokens, hkv, d)
        if c["rotary"]:
            s["q"] = normal(tokens, c["hq"], d)
            s["inv_freq"], s["mscale"] = _frequencies(c, dev)
    else:
        s["q"] = normal(tokens, c["hq"], d)
    return s


# ------------------------------------------------------------ plain forms
def _turn(x, pos, inv_freq, mscale, interleaved):
    """x [T, H, D] rotated in 32 bits; the angles of far positions need 64."""
    a = pos.double()[:, None, None] * inv_freq
    cos, sin = (a.cos() * mscale).float(), (a.sin() * mscale).float()
    r = 2 * inv_freq.numel()
    x = x.float()
    if interleaved:
        x1, x2 = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1).flatten(-2)
    else:
        x1, x2 = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1)
    return torch.cat((y, x[..., r:]), -1)


def _plain_rope(s):
    f = s["inv_freq"], s["mscale"], s["case"]["interleaved"]
    return (_turn(s["q"], s["pos"], *f).to(s["q"].dtype), _turn(s["k"], s["pos"], *f).to(s["k"].dtype))


def _places(s):
    """Each new token's sequence and position."""
    t = torch.arange(s["k_new" if "k_new" in s else "q"].shape[0], device=s["cu_q"].device)
    seq = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    return seq, s["kv_lens"].long()[seq] - s["cu_q"].long()[seq + 1] + t


def _plain_append(s):
    c = s["case"]
    seq, pos = _places(s)
    page, slot = s["table"].long()[seq, pos // c["page"]], pos % c["page"]
    k, v, d = s["k_new"].float(), s["v_new"].float(), c["dim"]
    out = {"k": s["k"], "v": s["v"]}
    if c["rotary"]:
        f = s["inv_freq"], s["mscale"], c["interleaved"]
        k = _turn(s["k_new"], pos, *f)
        out["q"] = _turn(s["q"], pos, *f).to(s["q"].dtype)
    if c["q8"]:
        x = k - s["k_mean"][:, :d]
        top = x.abs().amax(-1, keepdim=True)
        most = torch.full_like(top, 127.0)     # divided as tensors: one rounding each
        k = torch.where(top > 0, torch.round(x * (most / top)), 0.0)
        inv = torch.where(s["v_scale"] > 0, 1.0 / s["v_scale"], 0.0)[:, :d]
        v = (v * inv).clamp(-448, 448)
        s["k_scale"].transpose(1, 2)[page, slot] = (top / most).squeeze(-1)
        out["k_scale"] = s["k_scale"]
    at = (lambda x: x) if c["layout"] == "NHD" else (lambda x: x.transpose(1, 2))
    at(s["k"])[page, slot] = k.to(s["k"].dtype)
    at(s["v"]).view(torch.uint8 if c["q8"] else s["v"].dtype)[page, slot] = (
        v.to(s["v"].dtype).view(torch.uint8) if c["q8"] else v.to(s["v"].dtype))
    return out


def _plain_attn(s):
    c = s["case"]
    dev = s["q"].device
    hq, hkv, d, page = c["hq"], c["hkv"], c["dim"], c["page"]
    j = torch.arange(s["max_kv"], device=dev)
    pages, slots = s["table"].long()[:, j // page], (j % page).expand(c["n"], -1)
    at = (lambda x: x) if c["layout"] == "NHD" else (lambda x: x.transpose(1, 2))
    if c["q8"]:
        k = at(s["k"])[pages, slots].float() * s["k_scale"].transpose(1, 2)[pages, slots][..., None]
        v = at(s["v"]).view(torch.uint8)[pages, slots].view(torch.float8_e4m3fn).float()
        v = v * s["v_scale"][:, :d]
    else:
        k, v = at(s["k"])[pages, slots].float(), at(s["v"])[pages, slots].float()
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
        s["cache"] = sage.PagedCache(s["k"], s["v"], s["case"]["layout"], k_scale=s.get("k_scale"),
                                     k_mean=s.get("k_mean"), v_scale=s.get("v_scale"))
        s["batch"] = sage.PagedBatch(s["cu_q"], s["kv_lens"], s["table"], s["max_q"], s["max_kv"])
        s["ws"] = sage.alloc_workspace_paged()
    return s["cache"], s["batch"], s["ws"]


def _own_rope(s):
    from quantized_attention_smooth_gb300 import sage
    return sage.rope(s["q"], s["k"], s["pos"], s["inv_freq"], interleaved=s["case"]["interleaved"],
                     mscale=s["mscale"])


def _own_append(s):
    from quantized_attention_smooth_gb300 import sage
    c = s["case"]
    cache, batch, ws = _own_cache(sage, s)
    out = {"k": s["k"], "v": s["v"]}
    if c["rotary"]:
        out["q"] = sage.kv_append(cache, batch, s["k_new"], s["v_new"], q=s["q"],
                                  inv_freq=s["inv_freq"], interleaved=c["interleaved"],
                                  mscale=s["mscale"], ws=ws)
    else:
        sage.kv_append(cache, batch, s["k_new"], s["v_new"], ws=ws)
    if c["q8"]:
        out["k_scale"] = s["k_scale"]
    return out


def _own_attn(s):
    from quantized_attention_smooth_gb300 import sage
    cache, batch, ws = _own_cache(sage, s)
    return sage.attn_paged(cache, batch, s["q"], window=s["case"]["window"],
                           sinks=s["case"]["sinks"], ws=ws)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "attn": _own_attn}[op](state)
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn}[op](state)


# ------------------------------------------------------------- definition
def _exact_turn(x, pos, f, gain, interleaved):
    """Rotation of each channel pair as a product of complex numbers, in 64 bits."""
    x = x.double().clone()
    half = f.numel()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (
        slice(0, half), slice(half, 2 * half))
    turn = torch.polar(torch.full_like(pos.double()[:, None] * f, gain), pos.double()[:, None] * f)
    z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
    x[..., a], x[..., b] = z.real, z.imag
    return x


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        return tuple(_exact_turn(s[n], s["pos"], s["inv_freq"], s["mscale"], c["interleaved"])
                     for n in ("q", "k"))
    q_len, kv_len = _lens(c)
    d, hkv, page, group = c["dim"], c["hkv"], c["page"], c["hq"] // c["hkv"]
    start = 0
    if c["op"] == "append":
        nhd = c["layout"] == "NHD"
        k, v = s["k"].double(), s["v"].double()
        scale = s["k_scale"].double() if c["q8"] else None
        qs = []
        for i, (a, b) in enumerate(zip(q_len, kv_len)):
            pos = torch.arange(b - a, b, device=k.device)
            kn, vn = s["k_new"][start:start + a].double(), s["v_new"][start:start + a].double()
            if c["rotary"]:
                f = s["inv_freq"], s["mscale"], c["interleaved"]
                kn = _exact_turn(kn, pos, *f)
                qs.append(_exact_turn(s["q"][start:start + a], pos, *f))
            pg, sl = s["table"][i].long()[pos // page], pos % page
            if c["q8"]:
                off = (kn - s["k_mean"][:, :d].double()).abs().amax(-1)
                scale[pg, :, sl] = off / 127
                vn = (vn / s["v_scale"][:, :d].double()).clamp(-448, 448)
            if nhd:
                k[pg, sl], v[pg, sl] = kn, vn
            else:
                k[pg, :, sl], v[pg, :, sl] = kn, vn
            start += a
        out = {"k": None if c["q8"] else k, "v": v}
        if c["rotary"]:
            out["q"] = torch.cat(qs)
        if c["q8"]:
            out["k_scale"] = scale
        return out
    if work(c)["flops"] > 5e12:
        return None
    out = torch.zeros(sum(q_len), c["hq"], d, dtype=torch.float64, device=s["q"].device)
    for i, (a, b) in enumerate(zip(q_len, kv_len)):
        pages = s["table"][i, :-(-b // page)].long()
        pos = torch.arange(b - a, b, device=pages.device)[:, None]
        key = torch.arange(b, device=pages.device)[None]
        hidden = key > pos
        if c["window"] > 0:
            hidden |= (key <= pos - c["window"]) & (key >= c["sinks"])
        for h in range(hkv):
            if c["layout"] == "NHD":
                kh, vh = s["k"][pages, :, h].double(), s["v"][pages, :, h].double()
            else:
                kh, vh = s["k"][pages, h].double(), s["v"][pages, h].double()
            if c["q8"]:
                kh = kh * s["k_scale"][pages, h].double()[..., None]
                vh = vh * s["v_scale"][h, :d].double()
            kh, vh = kh.reshape(-1, d)[:b], vh.reshape(-1, d)[:b]
            for r in range(group):
                x = s["q"][start:start + a, h * group + r].double() @ kh.T * (d ** -0.5)
                x = torch.softmax(x.masked_fill_(hidden, float("-inf")), -1)
                out[start:start + a, h * group + r] = x @ vh
        start += a
    return out
