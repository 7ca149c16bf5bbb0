"""An 8-bit key/value cache and the log probabilities of a step, as measurable cases.

Three operators that a serving loop runs beside those of the 16-bit cache:

* ``append``    per-head RMSNorm of q and k, the position rotation, and the write of
                k and v into a paged cache of 8-bit floats (e4m3) with a scale for each
                block of 16 tokens and head (kda_paged_append_q8)
* ``attn``      attention of the new tokens over that cache (kda_paged_attn_q8)
* ``logprobs``  log probabilities of given tokens, their ranks, the entropy of the
                distribution and its most likely tokens, from logits
                (kda_token_logprobs)

``run`` computes them in elementary torch operations, or, when ``own`` is true,
through the library's entry points.
"""

import math
import random

import torch

own = False

KIND = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
E4M3 = torch.float8_e4m3fn
BLOCK = 16  # tokens of a scale
LEAST = 2.0 ** -50  # of the scales; the largest is 2^50


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # one user, one token, a short context: the smallest call, latency only
        dict(name="attn_decode_1", op="attn", B=1, q_lo=1, q_hi=1, c_lo=777, c_hi=777, lens=1,
             Hq=16, Hkv=2, d=128, page=16, dtype="bf16", causal=True),
        # an ordinary decode batch: every request one token, contexts of any length
        dict(name="attn_decode_256", op="attn", B=256, q_lo=1, q_hi=1, c_lo=511, c_hi=8191,
             lens=2, Hq=32, Hkv=8, d=128, page=64, dtype="bf16", causal=True),
        # a speculative verify step: 7 drafts and the last token, long contexts
        dict(name="attn_verify_64x8", op="attn", B=64, q_lo=8, q_hi=8, c_lo=1000, c_hi=32760,
             lens=3, Hq=32, Hkv=4, d=128, page=32, dtype="bf16", causal=True),
        # one chunk of a long prompt over what earlier chunks left in the cache
        dict(name="attn_chunk_8k", op="attn", B=1, q_lo=8192, q_hi=8192, c_lo=24576, c_hi=24576,
             lens=4, Hq=32, Hkv=8, d=128, page=128, dtype="bf16", causal=True),
        # a mixed batch: decodes, short prompts and chunks together, three heads a group
        dict(name="attn_mixed_24", op="attn", B=24, q_lo=1, q_hi=2047, c_lo=0, c_hi=8000, lens=5,
             Hq=24, Hkv=8, d=64, page=16, dtype="bf16", causal=True),
        # a small batch with fp32 queries (parity runs, small models)
        dict(name="attn_f32_8", op="attn", B=8, q_lo=1, q_hi=301, c_lo=0, c_hi=2500, lens=6, Hq=8,
             Hkv=2, d=64, page=16, dtype="f32", causal=True),
        # the tokens of one decode step of 64 requests, each into a block that was begun before
        dict(name="append_decode_64", op="append", T=64, runs=64, lens=7, pad=0, Hq=32, Hkv=8,
             d=128, rot=128, page=64, dtype="bf16", mode="half", norm=True, far=65536),
        # a full prefill batch, part of each head rotated, neighbouring pairs
        dict(name="append_32k", op="append", T=32767, runs=9, lens=8, pad=0, Hq=32, Hkv=8, d=128,
             rot=64, page=64, dtype="bf16", mode="interleaved", norm=True, far=1 << 20),
        # the sampled tokens of a handful of users, with five alternatives
        dict(name="logprobs_4", op="logprobs", N=4, V=50257, dtype="bf16", top=5, scale=1.0,
             masked=0.0),
        # a decode step of 256 users at a temperature, twenty alternatives, a grammar's mask
        dict(name="logprobs_256", op="logprobs", N=256, V=131072, dtype="f32", top=20, scale=1.25,
             masked=0.3),
        # the scoring of prompts: every position's next token, an odd vocabulary
        dict(name="logprobs_2047", op="logprobs", N=2047, V=128001, dtype="bf16", top=1, scale=1.0,
             masked=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "logprobs"])
    if op == "attn":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        Hkv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        while Hkv * group > 32:
            group = max(1, group // 2)
        case = dict(op="attn", Hq=Hkv * group, Hkv=Hkv, d=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64, 128, 256]), dtype=dtype,
                    causal=rng.random() < 0.85, lens=rng.randrange(1 << 30))
        form = rng.choice(["decode", "verify", "chunk", "mixed"])
        big = 1 if dtype == "bf16" else 8
        if form == "decode":
            case.update(B=_log(rng, 1, 256 // big), q_lo=1, q_hi=1)
            far = _log(rng, 16, 8000 // big)
        elif form == "verify":
            n = rng.randint(2, 16)
            case.update(B=_log(rng, 1, 64 // big), q_lo=n, q_hi=n)
            far = _log(rng, 16, 16000 // big)
        elif form == "chunk":
            n = _log(rng, 17, 8192 // big)
            case.update(B=1, q_lo=n, q_hi=n)
            far = _log(rng, 16, 24000 // big)
        else:
            case.update(B=rng.randint(2, 24), q_lo=0, q_hi=_log(rng, 2, 1500 // big))
            far = _log(rng, 16, 8000 // big)
        case.update(c_lo=rng.randint(0, far), c_hi=far)
        return case
    if op == "append":
        d = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        T = _log(rng, 1, 32000)
        return dict(op="append", T=T, runs=_log(rng, 1, min(T, 256)),
                    lens=rng.randrange(1 << 30), pad=rng.choice([0, 0, rng.randint(0, T // 2)]),
                    Hq=Hkv * rng.choice([1, 2, 3, 4]), Hkv=Hkv, d=d, rot=rng.choice([0, d // 2, d]), page=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]) if Hkv < 8 else "bf16",
                    mode=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.8,
                    far=_log(rng, 65536, 1 << 20))
    dtype = rng.choice(["bf16", "f32"])
    return dict(op="logprobs", N=_log(rng, 1, 2000 if dtype == "bf16" else 1000),
                V=_log(rng, 1000, 131000), dtype=dtype, top=rng.choice([0, 1, 2, 5, 20, 33, 64]),
                scale=rng.choice([1.0, 0.5, 1.7]), masked=rng.choice([0.0, 0.0, 0.9]))


def _lengths(case):
    """(new tokens, cached tokens) of each request of an attn case."""
    r = random.Random(case["lens"])
    new = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    cached = [r.randint(case["c_lo"], case["c_hi"]) for _ in range(case["B"])]
    new[0] = max(new[0], 1)
    return new, cached


def _runs(case, seed):
    """(position, tokens) of each request of an append case; its tokens go to
    consecutive slots, from the position's place in its page on.  Sizes and places
    in a page are the case's, the pages before them the seed's."""
    r, rs, ps = random.Random(case["lens"]), random.Random(seed), case["page"]
    T, R = case["T"] - case["pad"], min(case["runs"], case["T"] - case["pad"])
    cuts = sorted(r.sample(range(1, T), R - 1)) if R > 1 else []
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [T])]
    return [(rs.randint(0, (case["far"] - n) // ps - 1) * ps + r.randrange(ps), n) for n in sizes]


def _seen(case):
    """(row, key) pairs that an attn case's mask lets through, per query head."""
    pairs = 0
    for n, c in zip(*_lengths(case)):
        pairs += n * c + (n * (n + 1) // 2 if case["causal"] else n * n)
    return pairs


def work(case):
    op = case["op"]
    if op == "attn":
        new, cached = _lengths(case)
        T = sum(new)
        # a request without new tokens reads nothing
        keys = sum(n + c for n, c in zip(new, cached) if n)
        blocks = sum(-(-(n + c) // BLOCK) for n, c in zip(new, cached) if n)
        pages = sum(-(-(n + c) // case["page"]) for n, c in zip(new, cached) if n)
        return {"bytes": 2 * keys * case["Hkv"] * case["d"] + 8 * blocks * case["Hkv"]
                + 2 * T * case["Hq"] * case["d"] * SIZE[case["dtype"]] + 4 * pages
                + 8 * case["B"] + 4,
                "flops": 4 * _seen(case) * case["Hq"] * case["d"]}
    if op == "append":
        T, Hq, Hkv, d = case["T"] - case["pad"], case["Hq"], case["Hkv"], case["d"]
        es = SIZE[case["dtype"]]
        blocks = -(-T // BLOCK)  # at least; a scale is read and written for each
        return {"bytes": T * ((2 * Hq + 2 * Hkv) * d * es + 2 * Hkv * d + 4 * case["rot"] + 8)
                + 16 * blocks * Hkv,
                "flops": T * (6 * (Hq + Hkv) + 4 * Hkv) * d}
    N, V, K = case["N"], case["V"], case["top"]
    return {"bytes": N * (V * SIZE[case["dtype"]] + 16 + 8 * K), "flops": 6 * N * V}


# ----------------------------------------------------------------------- inputs

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1009 + salt)
    return g


def _normal(shape, gen, dtype, std=1.0, most=None):
    """N(0, std^2) in dtype, drawn in pieces so that no large fp32 copy is made."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        part = flat[i:i + (1 << 26)]
        x = torch.randn(part.shape, generator=gen, device="cuda")
        if std != 1.0:
            x.mul_(std)
        part.copy_(x.clamp_(-most, most) if most else x)
    return out


def _cu(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cache(n_pages, page, Hkv, d, gen):
    """Keys and values as a cache holds them, [2, n_pages, page, Hkv, d], and
    their scales [2, n_pages, page / 16, Hkv]: blocks whose largest value is near
    the type's, of magnitudes that differ by a few powers of two."""
    pages = _normal((2, n_pages, page, Hkv, d), gen, E4M3, std=96.0, most=448.0)
    power = torch.randint(-7, -4, (2, n_pages, page // BLOCK, Hkv), generator=gen, device="cuda")
    return pages, torch.exp2(power.float() - 0.5 * (power == -5))


def prepare(case, seed):
    st = {"op": case["op"], "case": case}
    g = _gen(seed, 1)
    if case["op"] == "attn":
        new, cached = _lengths(case)
        ps, dt, T = case["page"], KIND[case["dtype"]], sum(new)
        total = [n + c for n, c in zip(new, cached)]
        pages = [-(-t // ps) for t in total]
        n_pages = max(1, sum(pages))
        # pages of a request lie anywhere in the pool
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros((case["B"], max(1, max(pages))), dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = order[at:at + n]
            at += n
        kv, scales = _cache(n_pages, ps, case["Hkv"], case["d"], g)
        st.update(q=_normal((T, case["Hq"], case["d"]), g, dt), k=kv[0], v=kv[1], ks=scales[0],
                  vs=scales[1], table=table, cu=_cu(new), kv=_ints(total), new=new, total=total,
                  out=torch.zeros((T, case["Hq"], case["d"]), dtype=dt, device="cuda"))
    elif case["op"] == "append":
        T, ps, dt, d, rot = case["T"], case["page"], KIND[case["dtype"]], case["d"], case["rot"]
        heads = case["Hq"] + 2 * case["Hkv"]
        pos, place, at = [], [], 0
        for start, n in _runs(case, seed):
            off = start % ps
            pos.extend(range(start, start + n))
            place.extend(range(at + off, at + off + n))
            at += -(-(off + n) // ps) * ps
        n_pages = at // ps
        # pages of a request lie anywhere in the pool; padded rows have no slot
        order = torch.randperm(n_pages, generator=g, device="cuda")
        place = torch.tensor(place, device="cuda")
        slot = torch.full((T,), -1, dtype=torch.int32, device="cuda")
        slot[:len(place)] = (order[place // ps] * ps + place % ps).to(torch.int32)
        pages, scales = _cache(n_pages, ps, case["Hkv"], d, g)
        # tokens' magnitudes differ, so that some blocks that were begun before outgrow
        # their scales
        size = torch.exp2(torch.randn((T, 1, 1), generator=g, device="cuda"))
        qkv = _normal((T, heads, d), g, dt)
        qkv *= size.to(dt)
        st.update(qkv=qkv, pos=_ints(pos + [0] * case["pad"]), slot=slot, pages=pages,
                  scales=torch.exp2(torch.ceil(torch.log2(scales))),
                  wq=1 + 0.1 * torch.randn(d, generator=g, device="cuda") if case["norm"] else None,
                  wk=1 + 0.1 * torch.randn(d, generator=g, device="cuda") if case["norm"] else None,
                  rope=_rope(case["far"], rot) if rot else None,
                  q=torch.zeros((T, case["Hq"], d), dtype=dt, device="cuda"))
    else:
        N, V, dt, K = case["N"], case["V"], KIND[case["dtype"]], case["top"]
        # logits of a trained model: a few likely tokens, a long tail
        logits = _normal((N, V), g, dt, std=3.0)
        tokens = torch.randint(0, V, (N,), generator=g, device="cuda")
        if case["masked"]:
            # what a grammar forbids is -inf; the tokens themselves are allowed
            for part, t in zip(logits.split(64), tokens.split(64)):
                hide = torch.rand(part.shape, generator=g, device="cuda") < case["masked"]
                hide.scatter_(1, t[:, None], False)
                part.masked_fill_(hide, float("-inf"))
        f32, i32 = (dict(dtype=t, device="cuda") for t in (torch.float32, torch.int32))
        st.update(logits=logits, tokens=tokens.to(torch.int32), lp=torch.zeros(N, **f32),
                  ent=torch.zeros(N, **f32), ranks=torch.zeros(N, **i32),
                  top_ids=torch.zeros((N, K), **i32), top_lp=torch.zeros((N, K), **f32))
    if own:
        import hybrid_linear_attention_delta_gb300 as kda
        if case["op"] == "attn":
            st["ws"] = kda.paged_workspace_for(st["q"].shape[0], case["Hq"], case["Hkv"], case["d"])
        else:
            st["ws"] = kda.paged_workspace_for()
    return st


def _rope(n, rot):
    """cos | sin of position times 10000^(-2i/rot), angles in 64 bits: [n, rot]."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2 * i / rot)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


# ------------------------------------------------------------------- plain forms

def _values(pages, scales):
    """What a cache's pages and scales stand for, in bf16 (which holds a product
    of an e4m3 value with a power of two)."""
    n = pages.shape
    x = pages.to(torch.bfloat16).view(*n[:2], n[2] // BLOCK, BLOCK, *n[3:])
    return (x * scales.to(torch.bfloat16)[:, :, :, None, :, None]).view(n)


def _rows_of(st, b, dtype):
    """Keys and values of request b, gathered from its pages: [Hkv, keys, d]."""
    n, ps = st["total"][b], st["k"].shape[1]
    ids = st["table"][b, :-(-n // ps)].long()
    rows = []
    for pages, scales in ((st["k"], st["ks"]), (st["v"], st["vs"])):
        x = pages.view(torch.uint8)[ids].view(E4M3).to(dtype).flatten(0, 1)[:n]
        rows.append((x * scales[ids].to(dtype).flatten(0, 1).repeat_interleave(BLOCK, 0)[:n, :, None])
                    .permute(1, 0, 2))
    return rows


def _attend(st, dtype, budget):
    """Softmax attention, request by request, in blocks of query rows."""
    c = st["case"]
    Hkv, d, group = c["Hkv"], c["d"], c["Hq"] // c["Hkv"]
    out = torch.empty(st["q"].shape, dtype=dtype, device="cuda")
    t0 = 0
    for b, n in enumerate(st["new"]):
        if n == 0:
            continue
        keys = st["total"][b]
        k, v = _rows_of(st, b, dtype)
        step = max(1, budget // (c["Hq"] * keys))
        for a in range(0, n, step):
            m = min(step, n - a)
            q = st["q"][t0 + a:t0 + a + m].to(dtype).view(m, Hkv, group, d)
            q = q.permute(1, 0, 2, 3).reshape(Hkv, m * group, d)
            s = torch.matmul(q, k.transpose(1, 2)) * (1.0 / math.sqrt(d))
            if c["causal"]:
                row = torch.arange(m * group, device="cuda") // group + (keys - n + a)
                late = torch.arange(keys, device="cuda")[None, :] > row[:, None]
                s = s.masked_fill(late, float("-inf"))
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
            o = o.view(Hkv, m, group, d).permute(1, 0, 2, 3).reshape(m, Hkv * group, d)
            out[t0 + a:t0 + a + m] = o
        t0 += n
    return out


def _turned(st, dtype, rope):
    """q, k and v of an append case, normed and rotated."""
    c = st["case"]
    Hq, Hkv, rot = c["Hq"], c["Hkv"], c["rot"]
    x = st["qkv"].to(dtype)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    made = []
    for t, w in ((q, st["wq"]), (k, st["wk"])):
        if w is not None:
            t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w.to(dtype)
        if rot:
            cs = rope[st["pos"].long()][:, None, :]
            cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
            if c["mode"] == "half":
                a, b = t[..., :rot // 2], t[..., rot // 2:rot]
                turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
            else:
                a, b = t[..., 0:rot:2], t[..., 1:rot:2]
                turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
            t = torch.cat([turned, t[..., rot:]], -1)
        made.append(t)
    return made[0], made[1], v


def _scale_for(amax):
    """The smallest power of two p with amax <= 448 p, within the scales' range."""
    m, e = torch.frexp(amax.float())  # amax = m 2^e, m in [1/2, 1): 448 = 0.875 * 2^9
    power = torch.where(m <= 0.875, e - 9, e - 8).clamp(-50, 50)
    return torch.where(amax > 0, ((power + 127) << 23).view(torch.float32), LEAST)


def _append(st):
    """Scales grow with what comes into their block and start anew with a block's
    first token; what the block held before is rounded again where its scale grew."""
    q, k, v = _turned(st, torch.float32, st["rope"])
    real = torch.nonzero(st["slot"] >= 0)[:, 0]
    slot = st["slot"][real].long()
    st["q"][real] = q[real].to(st["q"].dtype)
    Hkv, d = k.shape[1:]
    block, off = slot // BLOCK, slot % BLOCK
    for i, x in ((0, k[real]), (1, v[real])):
        rows = st["pages"][i].view(torch.uint8).view(-1, BLOCK, Hkv, d)
        scales = st["scales"][i].view(-1, Hkv)
        n = scales.shape[0]
        amax = x.new_zeros((n, Hkv)).index_reduce_(0, block, x.abs().amax(-1), "amax")
        first = torch.full((n,), BLOCK, device="cuda").index_reduce_(0, block, off, "amin")
        old = torch.where((first == 0)[:, None], 0.0, scales)
        new = torch.where((first < BLOCK)[:, None], torch.maximum(old, _scale_for(amax)), scales)
        # tokens before the new ones, where the scale grew
        grown = torch.nonzero(((new > old) & (first < BLOCK)[:, None]).any(-1) & (first > 0))[:, 0]
        held = rows[grown].view(E4M3).float()
        ratio = (old / new)[grown][:, None, :, None]
        again = (held * ratio).to(E4M3).view(torch.uint8)
        before = torch.arange(BLOCK, device="cuda")[None, :, None, None] < first[grown][:, None, None, None]
        rows[grown] = torch.where(before & (ratio != 1), again, rows[grown])
        y = (x / new[block][:, :, None]).clamp(-448, 448).to(E4M3)
        rows.view(-1, Hkv, d)[slot] = y.view(torch.uint8)
        scales.copy_(new)
    return st["q"], _values(st["pages"], st["scales"])


def _logprobs(st):
    c = st["case"]
    x = st["logits"].float()
    t = st["tokens"].long()[:, None]
    xt = x.gather(1, t)
    i = torch.arange(c["V"], device="cuda")[None, :]
    ranks = ((x > xt) | ((x == xt) & (i < t))).sum(-1)
    # values in order, equal ones by their index: one whole number for both
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7fffffff), bits) * (1 << 32) + ((1 << 31) - i)
    del bits
    best = torch.topk(key, c["top"], dim=-1).values if c["top"] else key[:, :0]
    del key
    ids = (1 << 31) - (best - (best >> 32 << 32))
    # (a sum of 10^5 terms beside a logarithm near 0: in 64 bits)
    x = (x - x.amax(-1, keepdim=True)).double() * c["scale"]
    e = torch.exp(x)
    total = e.sum(-1, keepdim=True)
    lse = torch.log(total)
    lp = x.gather(1, t) - lse
    top = x.gather(1, ids) - lse
    ent = lse[:, 0] - (e * x.masked_fill(x == float("-inf"), 0.0)).sum(-1) / total[:, 0]
    none = top == float("-inf")
    return (lp[:, 0].float(), ent.float(), ranks.to(torch.int32),
            ids.masked_fill(none, -1).to(torch.int32), top.float())


def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "attn":
        return _attend(st, torch.float32, 1 << 28).to(st["out"].dtype)
    if st["op"] == "append":
        return _append(st)
    return _logprobs(st)


def _run_own(st):
    import hybrid_linear_attention_delta_gb300 as kda
    if st["op"] == "attn":
        kda.kda_paged_attn_q8(st["q"], st["k"], st["v"], st["ks"], st["vs"], st["table"], st["cu"],
                              st["kv"], st["out"], causal=st["case"]["causal"], workspace=st["ws"])
        return st["out"]
    if st["op"] == "append":
        pages, scales = st["pages"], st["scales"]
        kda.kda_paged_append_q8(st["qkv"], st["wq"], st["wk"], st["rope"], st["pos"], st["slot"],
                                st["q"], pages[0], pages[1], scales[0], scales[1],
                                rope_mode=st["case"]["mode"], norm_eps=1e-6, workspace=st["ws"])
        return st["q"], _values(pages, scales)
    kda.kda_token_logprobs(st["logits"], st["tokens"], st["lp"], st["ent"], st["ranks"],
                           st["top_ids"], st["top_lp"], scale=st["case"]["scale"],
                           workspace=st["ws"])
    return st["lp"], st["ent"], st["ranks"], st["top_ids"], st["top_lp"]


# ------------------------------------------------------------------------- exact

def exact(case, seed):
    """The operators' definitions in 64 bits, written apart from the plain forms:
    attention by a running maximum and sum over blocks of keys, the rotation as a
    complex product, 8-bit rounding by its grid, log probabilities row by row.
    Ranks and token numbers are whole and have no such value."""
    if case["op"] == "attn":
        # fp64 products run at about a teraflop a second
        if 4 * _seen(case) * case["Hq"] * case["d"] > 6e12:
            return None
        return _exact_attn(prepare(case, seed))
    if case["op"] == "append":
        return _exact_append(prepare(case, seed))
    st = prepare(case, seed)
    N, K = case["N"], case["top"]
    f64 = dict(dtype=torch.float64, device="cuda")
    lp, ent, top = torch.empty(N, **f64), torch.empty(N, **f64), torch.empty((N, K), **f64)
    rows = max(1, (1 << 26) // case["V"])
    for a in range(0, N, rows):
        y = st["logits"][a:a + rows].double() * case["scale"]
        p = torch.softmax(y, -1)
        z = torch.logsumexp(y, -1, keepdim=True)
        t = st["tokens"][a:a + rows].long()
        lp[a:a + rows] = y[torch.arange(len(y), device="cuda"), t] - z[:, 0]
        ent[a:a + rows] = (p * torch.where(p > 0, z - y, 0.0)).sum(-1)
        if K:
            top[a:a + rows] = torch.sort(y, -1, descending=True).values[:, :K] - z
    return lp, ent, None, None, top


def _nearest_e4m3(x):
    """x rounded to the nearest multiple of its e4m3 step (ties to even), at most 448."""
    power = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6.0)
    step = torch.exp2(power - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_append(st):
    case = st["case"]
    Hq, Hkv, rot, d = case["Hq"], case["Hkv"], case["rot"], case["d"]
    x = st["qkv"].double()
    res = []
    for t, w in ((x[:, :Hq], st["wq"]), (x[:, Hq:Hq + Hkv], st["wk"])):
        if w is not None:
            t = t * torch.rsqrt(t.square().sum(-1, keepdim=True) / d + 1e-6) * w.double()
        t = t.clone()
        if rot:
            cs = st["rope"].double()[st["pos"].long()]
            turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None]
            half = case["mode"] == "half"
            ia = torch.arange(rot // 2, device="cuda") * (1 if half else 2)
            ib = ia + (rot // 2 if half else 1)
            z = torch.complex(t[..., ia], t[..., ib]) * turn
            t[..., ia], t[..., ib] = z.real, z.imag
        res.append(t)
    n = case["T"] - case["pad"]
    q = st["q"].double()
    q[:n] = res[0][:n]
    slot = st["slot"][:n].long()
    values = []
    for i, t in ((0, res[1]), (1, x[:, Hq + Hkv:])):
        held = st["pages"][i].double().view(-1, BLOCK, Hkv, d)
        scale = st["scales"][i].double().view(-1, Hkv).clone()
        new = torch.full((held.shape[0] * BLOCK, Hkv, d), math.nan, dtype=torch.float64,
                         device="cuda")
        new[slot] = t[:n]
        new = new.view(held.shape)
        comes = ~torch.isnan(new[..., 0, 0])  # [blocks, 16]
        touched, starts = comes.any(1), comes[:, 0]
        largest = new.abs().nan_to_num(nan=0.0).amax((1, 3))
        power = torch.ceil(torch.log2(largest.clamp(min=1e-300) / 448.0)) - 1
        # (a logarithm may miss a whole number by its last bit)
        power = (power + (448.0 * torch.exp2(power) < largest)).clamp(-50.0, 50.0)
        grown = torch.where(starts[:, None], torch.exp2(power), torch.maximum(scale, torch.exp2(power)))
        grown = torch.where(touched[:, None], grown, scale)
        before = (comes.cumsum(1) == 0) & touched[:, None]
        wide = grown[:, None, :, None]
        again = _nearest_e4m3(held * scale[:, None, :, None] / wide)
        held = torch.where(before[..., None, None], again, held)
        held = torch.where(comes[..., None, None], _nearest_e4m3(new.nan_to_num(nan=0.0) / wide), held)
        values.append((held * wide).view(st["pages"][i].shape))
    return q, torch.stack(values)


def _exact_attn(st):
    c = st["case"]
    ps, Hkv, d, group = c["page"], c["Hkv"], c["d"], c["Hq"] // c["Hkv"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    block = 2048
    t0 = 0
    for b, n in enumerate(st["new"]):
        total = st["total"][b]
        if n == 0:
            continue
        key = torch.arange(total, device="cuda")
        flat = st["table"][b].long()[key // ps] * ps + key % ps
        for h in range(Hkv):
            K, W = (pages.view(torch.uint8).view(-1, Hkv, d)[flat, h].view(E4M3).double()
                    * scales.view(-1, Hkv)[flat // BLOCK, h, None].double()
                    for pages, scales in ((st["k"], st["ks"]), (st["v"], st["vs"])))
            for a in range(0, n, block):
                m = min(block, n - a)
                Q = st["q"][t0 + a:t0 + a + m, h * group:(h + 1) * group].double() / d ** 0.5
                Q = Q.reshape(m * group, d)
                last = total - n + a + torch.arange(m, device="cuda").repeat_interleave(group)
                if not c["causal"]:
                    last = torch.full_like(last, total - 1)
                top = torch.full((m * group,), -math.inf, dtype=torch.float64, device="cuda")
                den = torch.zeros_like(top)
                acc = torch.zeros((m * group, d), dtype=torch.float64, device="cuda")
                for j in range(0, total - n + a + m if c["causal"] else total, block):
                    S = Q @ K[j:j + block].T
                    S[key[None, j:j + block] > last[:, None]] = -math.inf
                    now = torch.maximum(top, S.max(-1).values)
                    E = torch.exp(S - now[:, None])
                    keep = torch.exp(top - now)
                    den = den * keep + E.sum(-1)
                    acc = acc * keep[:, None] + E @ W[j:j + block]
                    top = now
                out[t0 + a:t0 + a + m, h * group:(h + 1) * group] = \
                    (acc / den[:, None]).view(m, group, d)
        t0 += n
    return out
