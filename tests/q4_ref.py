"""The 4-bit cache's definition in plain torch, and small problems over it."""
import torch

from tests.paged_ref import HALF, Problem

GROUP = 32
SEVENTH = 0.14285714924335479736328125       # fl(1/7)
MOST_K, MOST_V = 9352.0, 1.0


def quantise(x, most):
    """x (..., D) float32 -> (codes -7..7 as int8 (..., 32 G), scales fp16 (..., G)); one IEEE
    operation a step, as the kernels take them."""
    d = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, -d % GROUP))
    parts = x.unflatten(-1, (-1, GROUP))
    s = (parts.abs().amax(-1) * SEVENTH).clamp(max=most).half()
    w = s.float()
    inv = torch.where(w > 0, torch.ones_like(w) / w, 0.0)
    n = torch.round(parts * inv[..., None]).clamp(-7, 7).to(torch.int8)
    return n.flatten(-2), s


def pack(n):
    u = (n + 8).to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def unpack(b):
    """Codes -8..7 of packed bytes, as int8."""
    return torch.stack(((b & 15).to(torch.int8) - 8, (b >> 4).to(torch.int8) - 8), -1).flatten(-2)


class Problem4(Problem):
    """A 4-bit cache with its batch."""

    def __init__(self, q_lens, kv_lens, hq, hkv, d, page, layout="NHD", q_dtype=torch.bfloat16,
                 window=0, sinks=0, seed=0, spare_rows=0, both=False, poison=True, dev="cuda",
                 pool=None, max_kv=None, offset=0.0, flat=False):
        super().__init__(q_lens, kv_lens, hq, hkv, d, page, layout, "q8", q_dtype, window, sinks,
                         seed, spare_rows, False, False, dev, pool, max_kv, offset)
        self.kind, self.k_scale = "q4", None
        g = torch.Generator(device=dev).manual_seed(seed + 77)
        pages, dp, groups = self.k.shape[0], 64 if d <= 64 else 128, -(-d // GROUP)
        self.groups = groups
        shape = (pages, page, hkv, 16 * groups) if layout == "NHD" else (pages, hkv, page, 16 * groups)
        tall = (pages, 2) + shape[1:] if both else (2,) + shape
        both_kv = torch.randint(0, 256, tall, generator=g, device=dev, dtype=torch.uint8)
        # the lowest code, 0, stands for -8: no writer makes it, yet it is a number
        self.k, self.v = (both_kv[:, 0], both_kv[:, 1]) if both else (both_kv[0], both_kv[1])
        one = lambda: torch.rand(pages, hkv, page, dp // GROUP, generator=g, device=dev)
        self.k_groups = ((one() + 0.3) * 0.2).half()
        self.v_groups = (one() * (0.0 if flat else 1.0)).half()
        self.k_groups[..., groups:] = float("nan")           # behind D: never used
        self.v_groups[..., groups:] = float("nan")
        self.v_scale = (torch.rand(hkv, dp, generator=g, device=dev) + 0.5) / 200
        if poison:
            self._poison4()

    def _poison4(self):
        """NaN scales where no new token sees a key; garbage table entries of unseen pages."""
        seen = torch.zeros(self.k.shape[0], self.page, dtype=torch.bool, device=self.q.device)
        for i, l in enumerate(self.kv_lens):
            if l == 0:
                continue
            any_row = self.visible(i).any(0) if self.q_lens[i] else torch.zeros(
                l, dtype=torch.bool, device=self.q.device)
            j = torch.arange(l, device=self.q.device)
            seen[self.table[i].long()[j // self.page], j % self.page] = any_row
            for s in range(-(-l // self.page)):
                if not any_row[s * self.page:(s + 1) * self.page].any():
                    self.table[i, s] = -7 if s % 2 else 2 ** 30 + 9
        for t in (self.k_groups, self.v_groups):
            t.masked_fill_(~seen[:, None, :, None], float("nan"))

    def rows(self, name, pages, slots):
        """Cached rows in 64 bits: (..., heads, D); K without its mean."""
        t = getattr(self, name)
        b = t[pages, slots] if self.layout == "NHD" else t[pages, :, slots]
        s = getattr(self, name + "_groups")[pages, :, slots][..., :self.groups].double()
        x = (unpack(b).double() * s.repeat_interleave(GROUP, -1))[..., :self.d]
        return x if name == "k" else x * 64 * self.v_scale[:, :self.d].double()

    def keys(self, i):
        l = self.kv_lens[i]
        j = torch.arange(l, device=self.q.device)
        pages = self.table[i].long()[j // self.page].clamp(0, self.k.shape[0] - 1)
        any_row = self.visible(i).any(0)[:, None, None]
        return tuple(torch.where(any_row, self.rows(n, pages, j % self.page), 0.0) for n in "kv")

    def bound(self, out, mean, spread, scale=None):
        """Elementwise bound on |kernel - reference|.  u |out|: the output's rounding.  P and P
        times the value's scale (or the value itself) are rounded to fp16, 2^-11 each; a key
        may be rounded to fp16 too, 2^-11 of each channel, which moves a logit by at most
        e = 2^-11 max_j sum |q k_j| scale (+ 2^-16 of fp32 sums, as |x| <= 40), and a weight by
        2 e relative.  Below 2^-14 fp16 has steps of 2^-24, half of one each for both
        roundings: of weights that are at least 2^7 at the largest, on values up to
        8 * 64 v_scale (code -8, scale 1)."""
        u = HALF[self.q.dtype]
        scale = self.d ** -0.5 if scale is None else scale
        e = torch.zeros_like(out[..., :1])
        most = torch.zeros_like(out)
        a = 0
        for i, n in enumerate(self.q_lens):
            if n and self.kv_lens[i]:
                k, _ = self.keys(i)
                for h in range(self.hq):
                    kh = k[:, h // (self.hq // self.hkv)].abs()
                    x = self.q[a:a + n, h].double().abs() @ kh.T * scale
                    e[a:a + n, h, 0] = x.amax(-1)
                    most[a:a + n, h] = (512 * self.v_scale[h // (self.hq // self.hkv), :self.d].double() *
                                        self.kv_lens[i])
            a += n
        e = (2.0 ** -11 + 3 * 2.0 ** -16) * e + 2.0 ** -16
        step = 2.0 ** -25 if self.q.dtype == torch.float16 else 1e-30
        return (u * out.abs() + (2 * 2.0 ** -11 + 2 * e * (1 + e)) * mean * (1 + u) * 1.01 +
                most * 2.0 ** -31 + step)

    def sage(self, sage):
        return (sage.PagedCache(self.k, self.v, self.layout, k_mean=self.k_mean,
                                v_scale=self.v_scale, k_groups=self.k_groups,
                                v_groups=self.v_groups, head_dim=self.d),
                sage.PagedBatch(self.cu, self.lens, self.table, self.max_q, self.max_kv))
