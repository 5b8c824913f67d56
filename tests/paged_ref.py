"""Plain 64-bit forms of the serving operators and small random problems for
their tests.  Cache slots that no new token may see hold NaN (or the scale NaN),
and block table entries without a visible key hold garbage page numbers."""
import torch

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # half a step, relative


def turn(x, pos, inv_freq, interleaved=False, gain=1.0, sign=1.0):
    """x (T, H, D) rotated in 64 bits."""
    x = x.double().clone()
    r = 2 * inv_freq.numel()
    a = pos.double()[:, None, None] * inv_freq.double().to(x.device) * sign
    c, s = a.cos() * gain, a.sin() * gain
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    x1, x2 = x[..., i].clone(), x[..., j].clone()
    x[..., i], x[..., j] = x1 * c - x2 * s, x2 * c + x1 * s
    return x


class Problem:
    """A paged cache with its batch.  q_lens and kv_lens per sequence; kind
    "f16", "bf16" or "q8"."""

    def __init__(self, q_lens, kv_lens, hq, hkv, d, page, layout="NHD", kind="bf16",
                 q_dtype=torch.bfloat16, window=0, sinks=0, seed=0, spare_rows=0, both=False,
                 poison=True, dev="cuda", pool=None, max_kv=None, offset=0.0):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.q_lens, self.kv_lens, self.hq, self.hkv, self.d = q_lens, kv_lens, hq, hkv, d
        self.page, self.layout, self.kind, self.window, self.sinks = page, layout, kind, window, sinks
        n = len(q_lens)
        used = [-(-x // page) for x in kv_lens]
        pool = pool or sum(used) + 2
        order = torch.randperm(pool, generator=g, device=dev)[:sum(used)]
        width = max(1, max(used)) + 1
        self.table = torch.full((n, width), 2 ** 30 + 5, dtype=torch.int32, device=dev)
        at = 0
        for i, u in enumerate(used):
            self.table[i, :u] = order[at:at + u].int()
            at += u
        cu = [0]
        for x in q_lens:
            cu.append(cu[-1] + x)
        self.cu = torch.tensor(cu, dtype=torch.int32, device=dev)
        self.lens = torch.tensor(kv_lens, dtype=torch.int32, device=dev)
        self.max_q, self.max_kv = max(q_lens), max_kv or max(1, max(kv_lens))
        self.q = torch.randn(cu[-1] + spare_rows, hq, d, generator=g, device=dev).to(q_dtype)
        shape = (pool, page, hkv, d) if layout == "NHD" else (pool, hkv, page, d)
        tall = (pool, 2) + shape[1:] if both else (2,) + shape
        kv = torch.randn(*tall, generator=g, device=dev)
        kf, vf = (kv[:, 0], kv[:, 1]) if both else (kv[0], kv[1])
        self.k_scale = self.k_mean = self.v_scale = None
        dp = 64 if d <= 64 else 128
        if kind == "q8":
            self.k_scale = (torch.rand(pool, hkv, page, generator=g, device=dev) + 0.5) / 60
            self.v_scale = (torch.rand(hkv, dp, generator=g, device=dev) + 0.5) / 100
            self.k_mean = torch.randn(hkv, dp, generator=g, device=dev) * offset
            codes = (kv * 40).round().clamp(-127, 127).to(torch.int8)
            self.k = (codes[:, 0] if both else codes[0])
            eight = (kv * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
            self.v = (eight[:, 1] if both else eight[1])
        else:
            dt = torch.float16 if kind == "f16" else torch.bfloat16
            kv = kv.to(dt)
            self.k, self.v = (kv[:, 0], kv[:, 1]) if both else (kv[0], kv[1])
        if poison:
            self._poison()

    def visible(self, i):
        """(rows, keys) truth table of sequence i."""
        n, l = self.q_lens[i], self.kv_lens[i]
        pos = torch.arange(l - n, l, device=self.q.device)[:, None]
        key = torch.arange(l, device=self.q.device)[None]
        see = key <= pos
        if self.window > 0:
            see &= (key > pos - self.window) | (key < self.sinks)
        return see

    def _poison(self):
        """NaN where no new token sees a key; garbage table entries of unseen pages."""
        pool = self.k.shape[0]
        seen = torch.zeros(pool, self.page, dtype=torch.bool, device=self.q.device)
        for i, l in enumerate(self.kv_lens):
            if l == 0:
                continue
            any_row = self.visible(i).any(0) if self.q_lens[i] else torch.zeros(
                l, dtype=torch.bool, device=self.q.device)
            j = torch.arange(l, device=self.q.device)
            pages = self.table[i].long()[j // self.page]
            seen[pages, j % self.page] = any_row
            for s in range(-(-l // self.page)):
                if not any_row[s * self.page:(s + 1) * self.page].any():
                    self.table[i, s] = -7 if s % 2 else 2 ** 30 + 9
        bad = ~seen
        nhd = self.layout == "NHD"
        mask = bad[:, :, None, None] if nhd else bad[:, None, :, None]
        if self.kind == "q8":
            self.k_scale.masked_fill_(bad[:, None, :], float("nan"))
            self.v.view(torch.uint8).masked_fill_(mask, 0x7F)          # e4m3's NaN
        else:
            self.k.masked_fill_(mask, float("nan"))
            self.v.masked_fill_(mask, float("nan"))

    def keys(self, i):
        """Sequence i's K and V (keys, heads, D) in 64 bits; rows nobody sees are zero."""
        l = self.kv_lens[i]
        j = torch.arange(l, device=self.q.device)
        pages = self.table[i].long()[j // self.page].clamp(0, self.k.shape[0] - 1)
        slot = j % self.page
        at = (lambda x: x[pages, slot]) if self.layout == "NHD" else (lambda x: x[pages, :, slot])
        if self.kind == "q8":
            k = at(self.k).double() * self.k_scale[pages, :, slot].double()[..., None]
            v = at(self.v).double() * self.v_scale[:, :self.d].double()
        else:
            k, v = at(self.k).double(), at(self.v).double()
        any_row = self.visible(i).any(0)[:, None, None]
        return torch.where(any_row, k, 0.0), torch.where(any_row, v, 0.0)

    def reference(self, scale=None):
        """out, lse and the two sums the tolerance needs, all (rows, Hq, ...) in 64 bits."""
        t = self.q.shape[0]
        dev = self.q.device
        out = torch.zeros(t, self.hq, self.d, dtype=torch.float64, device=dev)
        lse = torch.full((t, self.hq), float("-inf"), dtype=torch.float64, device=dev)
        mean, spread = torch.zeros_like(out), torch.zeros_like(out)
        scale = self.d ** -0.5 if scale is None else scale
        a = 0
        for i, n in enumerate(self.q_lens):
            if n and self.kv_lens[i]:
                k, v = self.keys(i)
                see = self.visible(i)
                for h in range(self.hq):
                    kh, vh = k[:, h // (self.hq // self.hkv)], v[:, h // (self.hq // self.hkv)]
                    x = self.q[a:a + n, h].double() @ kh.T * scale
                    x = x.masked_fill(~see, float("-inf"))
                    top = x.amax(-1, keepdim=True)
                    top = torch.where(top == float("-inf"), 0.0, top)
                    p = (x - top).exp()
                    l = p.sum(-1, keepdim=True)
                    w = torch.where(l > 0, p / l, 0.0)
                    out[a:a + n, h] = w @ vh
                    mean[a:a + n, h] = w @ vh.abs()
                    spread[a:a + n, h] = see.double() @ vh.abs() / torch.where(l > 0, l, 1.0)
                    lse[a:a + n, h] = (top + l.log()).squeeze(-1)
            a += n
        return out, lse, mean, spread

    def tolerance(self, out, mean, spread):
        """Elementwise bound on |kernel - reference|.  With weights w_j:
        the output's rounding, u |out|; P's rounding to the type of the tensor
        instruction, up p_j each, up sum w_j |v_j|; fp16's P below 2^-14 has
        steps of 2^-24, half of one each: 2^-25 sum |v_j| / l (l the sum of
        exponentials, P <= 1); an fp16 output below 2^-14 has the same steps, so its
        rounding is off by up to 2^-25 there.  The logits: |x| <= 40 here, with D <= 128 fp32
        products whose errors add up to less than 2^-16, which moves a weight
        by 2 * 2^-16 relative; the fp32 sums and exp2 stay below 2^-16 more."""
        u = HALF[self.q.dtype]
        up = 2.0 ** -8 if self.kind == "bf16" else 2.0 ** -11
        sub = 0.0 if self.kind == "bf16" else 2.0 ** -25
        step = 2.0 ** -25 if self.q.dtype == torch.float16 else 1e-30
        return u * out.abs() + (up + 3 * 2.0 ** -16) * mean * (1 + u) + sub * spread + step

    def sage(self, sage):
        return (sage.PagedCache(self.k, self.v, self.layout, self.k_scale, self.k_mean,
                                self.v_scale),
                sage.PagedBatch(self.cu, self.lens, self.table, self.max_q, self.max_kv))
