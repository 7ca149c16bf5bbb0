"""The 8-bit cache of the paged calls in plain 64-bit form, and its inputs: pages of
e4m3 values with a scale for 16 tokens and head."""

from __future__ import annotations

import torch

from paged_cases import BF16, F32, AttnCase, half_step

E4M3 = torch.float8_e4m3fn
NAN8 = 0x7f          # the byte of an e4m3 NaN
BLOCK = 16


def spread(scales):
    """A block's scale for each of its tokens: [..., pages, page, Hkv, 1]."""
    return scales.double().repeat_interleave(BLOCK, -2)[..., None]


class Q8AttnCase(AttnCase):
    """AttnCase over an 8-bit cache.  k and v are what the cache stands for, in 64
    bits; slots that belong to no key hold NaN, blocks without a key a NaN scale."""

    def __init__(self, new, total, *, dtype, powers=(-7, -5), seed=0, **kw):
        super().__init__(new, total, dtype=dtype, seed=seed, **kw)
        g = torch.Generator().manual_seed(seed + 77)
        for name in ("k", "v"):
            x = getattr(self, name).double()
            x = torch.where(x.abs() < 2.0 ** -6, torch.full_like(x, 2.0 ** -6).copysign(x), x)
            n_pages, page, Hkv, d = x.shape
            shape = (n_pages, page // BLOCK, Hkv)
            scales = torch.exp2(torch.randint(powers[0], powers[1] + 1, shape, generator=g).double()
                                + 0.3 * torch.rand(shape, generator=g).double()).float()
            pages = (x * 64).to(F32).to(E4M3)      # normal(0, 1): up to some 300
            used = ~torch.isnan(x[..., 0, 0]).view(n_pages, -1, BLOCK).all(-1)
            scales[~used] = float("nan")
            setattr(self, name + "8", pages)
            setattr(self, name + "_scales", scales)
            setattr(self, name, pages.double() * spread(scales))

    def set_values(self, name, x, scale):
        """The whole cache anew, with one scale."""
        pages = (x.double() / scale).to(F32).to(E4M3)
        setattr(self, name + "8", pages)
        s = torch.full((x.shape[0], x.shape[1] // BLOCK, x.shape[2]), scale)
        setattr(self, name + "_scales", s)
        setattr(self, name, pages.double() * spread(s))

    def bound(self, ref, size, top):
        """AttnCase.bound, and what the 8-bit cache adds.  fp32 queries: a key or a
        value times its scale is rounded once, a half step of sum |q k| and of the
        averaged |v|.  bf16 queries: a query's channels are scaled to at most 448 and
        split into two e4m3 parts, off by at most 2^-10 of those units, so by less than
        2^-17 of the row's largest channel (which is scaled to more than 128)."""
        u = half_step(F32)
        more = 2 * u * (max(top, 1.0) + 1)
        if self.dtype == BF16 and top > 0:
            live = torch.nan_to_num(self.k).abs().sum(-1).max()
            q = torch.nan_to_num(self.q.double()).abs().max()
            more += 2 * 2.0 ** -17 * float(q * live) * self.scale_used
        return super().bound(ref, size, top) + size * more

    def reference(self, causal=True, scale=None):
        self.scale_used = abs(self.d ** -0.5 if scale is None else scale)
        return super().reference(causal, scale)

    def cuda(self):
        names = ("q", "k8", "v8", "k_scales", "v_scales", "table", "cu", "kv")
        return {n: getattr(self, n).cuda() for n in names}


# ---------------------------------------------------------------------- append

def scale_for(amax):
    """The smallest power of two p in [2^-50, 2^50] with amax <= 448 p (64 bits)."""
    m, e = torch.frexp(amax.double())
    power = torch.where(m <= 0.875, e - 9, e - 8)
    power = torch.where(amax > 0, power, torch.full_like(power, -50)).clamp(-50, 50)
    return torch.exp2(power.double())


def rounded(x):
    """x rounded to e4m3 (ties to even), at most 448: in 64 bits, by its grid."""
    e = torch.frexp(x.abs())[1].clamp(min=-5) - 1         # |x| in [2^e, 2^(e+1))
    step = torch.exp2((e - 3).double())
    return (torch.round(x / step) * step).clamp(-448, 448)


def append_blocks(x, slots, pages, scales):
    """What an append leaves of one tensor: (values before the division by the
    scale, where they come, the scales of exact values, first new slot of a block).
    x [T, Hkv, d] in 64 bits, pages and scales as they were."""
    n_pages, page, Hkv, d = pages.shape
    n = n_pages * page // BLOCK
    new = torch.full((n, BLOCK, Hkv, d), float("nan"), dtype=torch.float64)
    first = torch.full((n,), BLOCK)
    comes = torch.zeros((n, BLOCK), dtype=torch.bool)
    for t, s in enumerate(slots.tolist()):
        if s < 0:
            continue
        new[s // BLOCK, s % BLOCK] = x[t]
        comes[s // BLOCK, s % BLOCK] = True
        first[s // BLOCK] = min(int(first[s // BLOCK]), s % BLOCK)
    return new, comes, first
