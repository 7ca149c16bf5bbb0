"""Plain 64-bit forms of the paged full-attention calls and of the draft
verification, for the tests (on the CPU, one request at a time), and the
inputs they are run on."""

from __future__ import annotations

import math

import torch

BF16, F32 = torch.bfloat16, torch.float32
DT = {"bf16": BF16, "f32": F32}


def half_step(dtype) -> float:
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------- attention

class AttnCase:
    """Requests over a shuffled page pool.  Slots that belong to no key hold
    NaN, unused block-table entries point at a page of NaNs, and token rows
    behind the last request are marked."""

    MARK = 7.0

    def __init__(self, new, total, *, Hq, Hkv, d, page, dtype, seed=0, pad=0, extra_pages=3,
                 scale_q=1.0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.total, self.dtype = list(new), list(total), DT[dtype]
        self.Hq, self.Hkv, self.d, self.page = Hq, Hkv, d, page
        T = sum(new)
        pages = [-(-t // page) for t in total]
        n_pages = sum(pages) + extra_pages
        order = torch.randperm(n_pages, generator=g)
        spare = int(order[-1]) if extra_pages else 0
        self.table = torch.full((len(new), max(1, max(pages, default=1))), spare,
                                dtype=torch.int32)
        self.k = torch.full((n_pages, page, Hkv, d), float("nan"), dtype=self.dtype)
        self.v = torch.full_like(self.k, float("nan"))
        at = 0
        for b, n in enumerate(pages):
            ids = order[at:at + n]
            self.table[b, :n] = ids.to(torch.int32)
            at += n
            for x in (self.k, self.v):
                rows = x[ids].reshape(n * page, Hkv, d)
                rows[:total[b]] = torch.randn((total[b], Hkv, d), generator=g).to(self.dtype)
                x[ids] = rows.reshape(n, page, Hkv, d)
        self.q = (scale_q * torch.randn((T + pad, Hq, d), generator=g)).to(self.dtype)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        self.cu = torch.tensor(cu, dtype=torch.int32)
        self.kv = torch.tensor(total, dtype=torch.int32)

    def reference(self, causal=True, scale=None):
        """(out, |v| averaged with the same weights, most of sum |q k| scale)."""
        c = self.d ** -0.5 if scale is None else scale
        G = self.Hq // self.Hkv
        out = torch.zeros(self.q.shape, dtype=torch.float64)
        size = torch.zeros_like(out)
        top = 0.0
        for b, (n, total) in enumerate(zip(self.new, self.total)):
            if n == 0 or total == 0:
                continue
            ids = self.table[b, :-(-total // self.page)].long()
            K = self.k[ids].flatten(0, 1)[:total].double()
            V = self.v[ids].flatten(0, 1)[:total].double()
            t0 = int(self.cu[b])
            for h in range(self.Hq):
                q = self.q[t0:t0 + n, h].double()
                s = c * (q @ K[:, h // G].T)
                top = max(top, abs(c) * float((q.abs() @ K[:, h // G].abs().T).max()))
                if causal:
                    pos = total - n + torch.arange(n)
                    s.masked_fill_(torch.arange(total)[None] > pos[:, None], -math.inf)
                m = s.max(-1, keepdim=True).values
                e = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
                z = e.sum(-1, keepdim=True)
                w = torch.where(z > 0, e / z, 0.0)
                out[t0:t0 + n, h] = w @ V[:, h // G]
                size[t0:t0 + n, h] = w @ V[:, h // G].abs()
        return out, size, top

    def bound(self, ref, size, top):
        """Largest error of each output.  bf16: the weights are rounded to bf16
        (half a step each, so at most that times the averaged |v|) and the
        output is rounded once.  Both: the score's d products are summed in
        fp32 (d half steps of sum |q k|, doubled for truncating adders), which
        moves a weight by that much relative, in the numerator and in the sum;
        the sums over the keys add at most a half step per key."""
        u = half_step(F32)
        keys = max(self.total, default=1)
        score = 2 * (self.d + 8) * u * max(top, 1.0)
        out = 2 * score + 4 * u * keys + 16 * u
        rel = half_step(self.dtype)
        weights = rel if self.dtype == BF16 else 0.0
        return rel * ref.abs() * 1.01 + size * (weights * 1.01 + out) + 1e-30

    def cuda(self):
        return {n: getattr(self, n).cuda() for n in ("q", "k", "v", "table", "cu", "kv")}


# ---------------------------------------------------------------------- append

def append_reference(qkv, q_norm, k_norm, rope, positions, Hq, Hkv, mode, eps):
    """(q, k, v) of every token in fp64, and for each the size of the terms that
    its rotation adds up (for the error bound)."""
    x = qkv.double()
    parts = []
    for t, w in ((x[:, :Hq], q_norm), (x[:, Hq:Hq + Hkv], k_norm)):
        if w is not None:
            t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps) * w.double()
        t = t.clone()
        size = t.abs()
        if rope is not None:
            rot = rope.shape[1]
            cs = rope.double()[positions.long()][:, None]
            c, s = cs[..., :rot // 2], cs[..., rot // 2:]
            a = (slice(0, rot // 2), slice(rot // 2, rot)) if mode == "half" else \
                (slice(0, rot, 2), slice(1, rot, 2))
            u, v = t[..., a[0]].clone(), t[..., a[1]].clone()
            size = size.clone()
            t[..., a[0]], t[..., a[1]] = u * c - v * s, u * s + v * c
            size[..., a[0]] = (u * c).abs() + (v * s).abs()
            size[..., a[1]] = (u * s).abs() + (v * c).abs()
        parts.append((t, size))
    return parts[0], parts[1], x[:, Hq + Hkv:]


# ------------------------------------------------------------------------ plan

def plan_reference(cu, cached, table, held, ring, head, count, page, T):
    """The page bookkeeping, request by request, on Python ints."""
    n_pages, B = len(ring), len(cached)
    table, ring_out = [list(r) for r in table], list(ring)
    width = len(table[0]) if B else 0
    taken = back = 0
    asked = 0
    held_out, kv, pos, slot = [], [], [0] * T, [-1] * T
    for b in range(B):
        total = cached[b] + cu[b + 1] - cu[b]
        ok = cached[b] >= 0 and 0 <= held[b] <= width and total <= width * page
        want = -(-total // page) if ok else held[b]
        need = max(0, want - held[b])
        asked += need
        if not ok or (need and asked > count):
            held_out.append(held[b])
            kv.append(0)
            continue
        for j in range(held[b], want):
            table[b][j] = ring[(head + taken) % n_pages]
            taken += 1
        for j in range(want, held[b]):
            if count + back < n_pages:
                ring_out[(head + count + back) % n_pages] = table[b][j]
                back += 1
        held_out.append(want)
        kv.append(total)
        for t in range(cu[b], cu[b + 1]):
            p = cached[b] + t - cu[b]
            pos[t], slot[t] = p, table[b][p // page] * page + p % page
    return dict(table=table, held_out=held_out, ring=ring_out,
                ring_out=[(head + taken) % n_pages, count - taken + back], kv=kv, positions=pos,
                slots=slot)


# ---------------------------------------------------------------------- verify

def verify_reference(p, q, x, ua, us, lens=None):
    """accepted, tokens in fp64, sequence by sequence."""
    N, n1, V = p.shape
    accepted, tokens = [], []
    for n in range(N):
        L = n1 - 1 if lens is None else int(lens[n])
        kept = 0
        while kept < L:
            t = int(x[n, kept])
            if not 0 <= t < V:
                break
            qx = 1.0 if q is None else float(q[n, kept, t])
            if not float(ua[n, kept]) * qx < float(p[n, kept, t]):
                break
            kept += 1
        r = p[n, kept].double()
        if kept < L:
            if q is not None:
                left = (r - q[n, kept].double()).clamp(min=0)
            else:
                left = r.clone()
                if 0 <= int(x[n, kept]) < V:
                    left[int(x[n, kept])] = 0
            if float(left.sum()) > 0:
                r = left
        cum = torch.cumsum(r, 0)
        at = int((cum <= float(us[n]) * float(cum[-1])).sum())
        accepted.append(kept + 1)
        tokens.append([int(t) for t in x[n, :kept]] + [min(at, V - 1)] + [-1] * (n1 - 1 - kept))
    return torch.tensor(accepted, dtype=torch.int32), torch.tensor(tokens, dtype=torch.int32)
