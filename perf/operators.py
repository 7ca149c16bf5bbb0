"""The full-attention side of a hybrid stack's serving step, as measurable cases.

Four operators that a serving loop runs beside the recurrent layers:

* ``plan``    pages, positions and cache slots of a step's new tokens, from the
              requests' lengths (kda_paged_plan)
* ``append``  per-head RMSNorm of q and k, the position rotation, and the write
              of k and v into the paged cache, from the packed projection
              (kda_paged_append)
* ``attn``    attention of the new tokens over the paged cache
              (kda_paged_attn)
* ``verify``  verification of drafted tokens against the target's
              probabilities with given random numbers (kda_verify_drafts)

``run`` computes them in elementary torch operations, or, when ``own`` is
true, through the library's entry points.
"""

import math
import random

import torch

own = False

KIND = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


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
        # a small fp32 batch (parity runs, small models)
        dict(name="attn_f32_8", op="attn", B=8, q_lo=1, q_hi=301, c_lo=0, c_hi=2500, lens=6, Hq=8,
             Hkv=2, d=64, page=16, dtype="f32", causal=True),
        # the tokens of one decode step of 64 requests
        dict(name="append_decode_64", op="append", T=64, Hq=32, Hkv=8, d=128, rot=128, page=64,
             dtype="bf16", mode="half", norm=True, far=65536),
        # a full prefill batch, part of each head rotated, neighbouring pairs
        dict(name="append_32k", op="append", T=32767, Hq=32, Hkv=8, d=128, rot=64, page=64,
             dtype="bf16", mode="interleaved", norm=True, far=1 << 20),
        # the page bookkeeping of a decode step
        dict(name="plan_decode_64", op="plan", B=64, n_lo=1, n_hi=1, c_lo=0, c_hi=16000, lens=7,
             page=64, spare=256),
        # a large mixed step: decodes, chunks and finished requests that give pages back
        dict(name="plan_mixed_2048", op="plan", B=2048, n_lo=0, n_hi=61, c_lo=0, c_hi=8000,
             lens=8, page=16, spare=20000),
        # three looked-up drafts (no draft probabilities) for a handful of users
        dict(name="verify_4x3", op="verify", N=4, n_draft=3, V=50257, dtype="bf16", probs=False),
        # the verify step's acceptance for 64 users, seven drafts each
        dict(name="verify_64x7", op="verify", N=64, n_draft=7, V=131072, dtype="f32", probs=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "plan", "verify"])
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
        return dict(op="append", T=_log(rng, 1, 32000), Hq=Hkv * rng.choice([1, 2, 3, 4]), Hkv=Hkv,
                    d=d, rot=rng.choice([0, d // 2, d]), page=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]) if Hkv < 8 else "bf16",
                    mode=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.8,
                    far=_log(rng, 4096, 1 << 20))
    if op == "plan":
        return dict(op="plan", B=_log(rng, 1, 2000), n_lo=0, n_hi=_log(rng, 1, 60),
                    c_lo=0, c_hi=_log(rng, 64, 8000), lens=rng.randrange(1 << 30),
                    page=rng.choice([16, 32, 64, 128]), spare=_log(rng, 4, 20000))
    dtype = rng.choice(["f32", "bf16"])
    return dict(op="verify", N=_log(rng, 1, 64), n_draft=rng.randint(0, 7),
                V=_log(rng, 1000, 131000), dtype=dtype, probs=rng.random() < 0.7)


def _lengths(case):
    """(new tokens, cached tokens) of each request of an attn case."""
    r = random.Random(case["lens"])
    new = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    cached = [r.randint(case["c_lo"], case["c_hi"]) for _ in range(case["B"])]
    new[0] = max(new[0], 1)
    return new, cached


def _plan_lengths(case):
    """(new tokens, cached tokens, pages held before) of each request; one
    request in 16 is finished (no tokens left) and gives its pages back."""
    r = random.Random(case["lens"])
    new, cached, held = [], [], []
    for _ in range(case["B"]):
        c = r.randint(case["c_lo"], case["c_hi"])
        h = -(-c // case["page"])
        if r.randrange(16) == 0:
            new.append(0), cached.append(0)
        else:
            new.append(r.randint(case["n_lo"], case["n_hi"])), cached.append(c)
        held.append(h)
    new[0] = max(new[0], 1)
    return new, cached, held


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
        es, T = SIZE[case["dtype"]], sum(new)
        # a request without new tokens reads nothing
        keys = sum(n + c for n, c in zip(new, cached) if n)
        pages = sum(-(-(n + c) // case["page"]) for n, c in zip(new, cached) if n)
        return {"bytes": (2 * keys * case["Hkv"] + 2 * T * case["Hq"]) * case["d"] * es
                + 4 * pages + 8 * case["B"] + 4,
                "flops": 4 * _seen(case) * case["Hq"] * case["d"]}
    if op == "append":
        heads = case["Hq"] + 2 * case["Hkv"]
        elems = case["T"] * heads * case["d"]
        return {"bytes": 2 * elems * SIZE[case["dtype"]] + case["T"] * (4 * case["rot"] + 8),
                "flops": 6 * case["T"] * (case["Hq"] + case["Hkv"]) * case["d"]}
    if op == "plan":
        new, cached, held = _plan_lengths(case)
        want = [-(-(n + c) // case["page"]) for n, c in zip(new, cached)]
        moved = sum(abs(w - h) for w, h in zip(want, held))
        return {"bytes": 20 * case["B"] + 8 * moved + 8 * sum(new) + 20, "flops": 4 * sum(new)}
    # one target row and one draft row of each sequence; the candidates' entries
    rows = 2 if case["probs"] and case["n_draft"] else 1
    row = rows * case["V"] * SIZE[case["dtype"]] + 32 * case["n_draft"] + 12
    return {"bytes": case["N"] * row, "flops": 3 * case["N"] * case["V"]}


# ----------------------------------------------------------------------- inputs

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1009 + salt)
    return g


def _normal(shape, gen, dtype):
    """N(0, 1) in dtype, drawn in pieces so that no large fp32 copy is made."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        part = flat[i:i + (1 << 26)]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
    return out


def _cu(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


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
        shape = (n_pages, ps, case["Hkv"], case["d"])
        st.update(q=_normal((T, case["Hq"], case["d"]), g, dt), k=_normal(shape, g, dt),
                  v=_normal(shape, g, dt), table=table, cu=_cu(new), kv=_ints(total), new=new,
                  total=total, out=torch.zeros((T, case["Hq"], case["d"]), dtype=dt, device="cuda"))
    elif case["op"] == "append":
        T, ps, dt, d, rot = case["T"], case["page"], KIND[case["dtype"]], case["d"], case["rot"]
        heads = case["Hq"] + 2 * case["Hkv"]
        # tokens of a step sit at consecutive positions, a run for each request
        r = random.Random(seed)
        pos, run = [], 0
        while len(pos) < T:
            run = min(T - len(pos), r.randint(1, max(1, T // 4)), case["far"])
            start = r.randint(0, case["far"] - run)
            pos.extend(range(start, start + run))
        n_pages = -(-T // ps) + 1
        order = torch.randperm(n_pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        st.update(qkv=_normal((T, heads, d), g, dt), pos=_ints(pos),
                  slot=(order[t // ps] * ps + t % ps).to(torch.int32),
                  wq=1 + 0.1 * torch.randn(d, generator=g, device="cuda") if case["norm"] else None,
                  wk=1 + 0.1 * torch.randn(d, generator=g, device="cuda") if case["norm"] else None,
                  rope=_rope(case["far"], rot) if rot else None,
                  q=torch.zeros((T, case["Hq"], d), dtype=dt, device="cuda"))
        shape = (n_pages, ps, case["Hkv"], d)
        st.update(k=torch.zeros(shape, dtype=dt, device="cuda"),
                  v=torch.zeros(shape, dtype=dt, device="cuda"))
    elif case["op"] == "plan":
        new, cached, held = _plan_lengths(case)
        ps, T = case["page"], sum(new)
        want = [-(-(n + c) // ps) for n, c in zip(new, cached)]
        need = sum(max(0, w - h) for w, h in zip(want, held))
        n_held, n_free = sum(held), need + case["spare"]
        n_pages = n_held + n_free
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        width = max(1, max(max(w, h) for w, h in zip(want, held)))
        table = torch.zeros((case["B"], width), dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(held):
            table[b, :n] = order[at:at + n]
            at += n
        ring = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        head = random.Random(seed).randrange(n_pages)
        where = (head + torch.arange(n_free, device="cuda")) % n_pages
        ring[where] = order[n_held:]
        st.update(cu=_cu(new), cached=_ints(cached), table=table, held=_ints(held), ring=ring,
                  state=_ints([head, n_free]), held_out=_ints([0] * case["B"]),
                  state_out=_ints([0, 0]), kv=_ints([0] * case["B"]),
                  pos=torch.zeros(T, dtype=torch.int32, device="cuda"),
                  slot=torch.zeros(T, dtype=torch.int32, device="cuda"), T=T, page=ps)
    else:
        N, n, V, dt = case["N"], case["n_draft"], case["V"], KIND[case["dtype"]]
        # logits of a trained model: a few likely tokens, a long tail; the draft
        # model's are the target's with noise
        logits = 3.0 * torch.randn((N, n + 1, V), generator=g, device="cuda")
        st["p"] = _softmax(logits).to(dt)
        noisy = logits[:, :n] + 0.7 * torch.randn((N, n, V), generator=g, device="cuda")
        del logits
        q = _softmax(noisy).to(dt)
        del noisy
        u = torch.rand((N, n, 1), generator=g, device="cuda")
        cum = torch.cumsum(q.float(), -1)
        st["x"] = (cum < u * cum[..., -1:]).sum(-1).clamp(max=V - 1).to(torch.int32)
        del cum
        st.update(q=q if case["probs"] and n else None,
                  ua=torch.rand((N, n), generator=g, device="cuda"),
                  us=torch.rand((N,), generator=g, device="cuda"),
                  accepted=torch.zeros(N, dtype=torch.int32, device="cuda"),
                  tokens=torch.zeros((N, n + 1), dtype=torch.int32, device="cuda"))
    if own:
        import hybrid_linear_attention_delta_gb300 as kda
        if case["op"] == "attn":
            st["ws"] = kda.paged_workspace_for(st["q"].shape[0], case["Hq"], case["Hkv"], case["d"])
        else:
            st["ws"] = kda.paged_workspace_for()
    return st


def _softmax(x):
    x = torch.exp(x - x.amax(-1, keepdim=True))
    return x / x.sum(-1, keepdim=True)


def _rope(n, rot):
    """cos | sin of position times 10000^(-2i/rot), angles in 64 bits: [n, rot]."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2 * i / rot)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


# ------------------------------------------------------------------- plain forms

def _rows_of(st, b, dtype):
    """Keys and values of request b, gathered from its pages: [Hkv, keys, d]."""
    n, ps = st["total"][b], st["k"].shape[1]
    ids = st["table"][b, :-(-n // ps)].long()
    return [st[name][ids].flatten(0, 1)[:n].to(dtype).permute(1, 0, 2) for name in ("k", "v")]


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


def _append(st, dtype, rope):
    c = st["case"]
    Hq, Hkv, d, rot = c["Hq"], c["Hkv"], c["d"], c["rot"]
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


def _plan(st):
    ps, table, ring = st["page"], st["table"], st["ring"]
    B, width = table.shape
    n_pages = ring.numel()
    cu, cached, held = st["cu"].long(), st["cached"].long(), st["held"].long()
    total = cached + cu[1:] - cu[:-1]
    want = (total + ps - 1) // ps
    need, back = (want - held).clamp(min=0), (held - want).clamp(min=0)
    head, count = st["state"][0].long(), st["state"][1].long()
    col = torch.arange(width, device="cuda")[None, :]
    # pages given back go behind the free ones, in request order
    first = torch.cumsum(back, 0) - back
    gone = (col >= want[:, None]) & (col < held[:, None])
    at = (head + count + first[:, None] + col - want[:, None]) % n_pages
    # (entries that are not given back are written to a spare place)
    spare = torch.cat([ring, ring.new_zeros(1)])
    spare[torch.where(gone, at, n_pages).flatten()] = table.flatten()
    # new pages come off the front
    first = torch.cumsum(need, 0) - need
    fresh = (col >= held[:, None]) & (col < want[:, None])
    at = (head + first[:, None] + col - held[:, None]) % n_pages
    table.copy_(torch.where(fresh, ring[at], table))
    ring.copy_(spare[:n_pages])
    taken = need.sum()
    state = torch.stack([(head + taken) % n_pages, count - taken + back.sum()]).to(torch.int32)
    t = torch.arange(st["T"], device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    pos = cached[b] + t - cu[b]
    slot = table[b, pos // ps] * ps + pos % ps
    return (table, want.to(torch.int32), ring, state, total.to(torch.int32), pos.to(torch.int32),
            slot.to(torch.int32))


def _verify(st):
    p, q, x = st["p"], st["q"], st["x"].long()
    N, n = x.shape
    V = p.shape[-1]
    rows = torch.arange(N, device="cuda")
    px = p[:, :n].gather(-1, x[..., None])[..., 0].double()
    qx = q.gather(-1, x[..., None])[..., 0].double() if q is not None else torch.ones_like(px)
    kept = (st["ua"].double() * qx < px).to(torch.int32).cumprod(-1).sum(-1)
    r = p[rows, kept].double()
    if n:
        stop = kept.clamp(max=n - 1)
        if q is not None:
            left = (r - q[rows, stop].double()).clamp(min=0)
        else:
            left = r.scatter(1, x[rows, stop][:, None], 0.0)
        # nothing left of the target after the subtraction: the target itself
        use = (kept < n) & (left.sum(-1) > 0)
        r = torch.where(use[:, None], left, r)
    cum = torch.cumsum(r, -1)
    chosen = (cum <= st["us"].double()[:, None] * cum[:, -1:]).sum(-1).clamp(max=V - 1)
    at = torch.arange(n + 1, device="cuda")[None, :]
    padded = torch.cat([x, x.new_zeros(N, 1)], 1)
    tokens = torch.where(at < kept[:, None], padded, torch.where(at == kept[:, None],
                                                                 chosen[:, None], -1))
    return (kept + 1).to(torch.int32), tokens.to(torch.int32)


def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "attn":
        return _attend(st, torch.float32, 1 << 28).to(st["out"].dtype)
    if st["op"] == "append":
        q, k, v = _append(st, torch.float32, st["rope"])
        slot = st["slot"].long()
        for pages, t in ((st["k"], k), (st["v"], v)):
            pages.view(-1, *pages.shape[2:])[slot] = t.to(pages.dtype)
        return q.to(st["q"].dtype), st["k"], st["v"]
    if st["op"] == "plan":
        return _plan(st)
    return _verify(st)


def _run_own(st):
    import hybrid_linear_attention_delta_gb300 as kda
    if st["op"] == "attn":
        kda.kda_paged_attn(st["q"], st["k"], st["v"], st["table"], st["cu"], st["kv"], st["out"],
                           causal=st["case"]["causal"], workspace=st["ws"])
        return st["out"]
    if st["op"] == "append":
        kda.kda_paged_append(st["qkv"], st["wq"], st["wk"], st["rope"], st["pos"], st["slot"],
                             st["q"], st["k"], st["v"], rope_mode=st["case"]["mode"],
                             norm_eps=1e-6, workspace=st["ws"])
        return st["q"], st["k"], st["v"]
    if st["op"] == "plan":
        kda.kda_paged_plan(st["cu"], st["cached"], st["table"], st["held"], st["ring"],
                           st["state"], st["held_out"], st["state_out"], st["kv"], st["pos"],
                           st["slot"], page_size=st["page"], workspace=st["ws"])
        return (st["table"], st["held_out"], st["ring"], st["state_out"], st["kv"], st["pos"],
                st["slot"])
    kda.kda_verify_drafts(st["p"], st["q"], st["x"], st["ua"], st["us"], st["accepted"],
                          st["tokens"], workspace=st["ws"])
    return st["accepted"], st["tokens"]


# ------------------------------------------------------------------------- exact

def exact(case, seed):
    """The operators' definitions in 64 bits, written apart from the plain
    forms: attention by a running maximum and sum over blocks of keys, the
    rotation as a complex product.  Plans and verified tokens are whole
    numbers and have no such value."""
    if case["op"] == "plan" or case["op"] == "verify":
        return None
    if case["op"] == "attn":
        # fp64 products run at about a teraflop a second
        if 4 * _seen(case) * case["Hq"] * case["d"] > 6e12:
            return None
        return _exact_attn(prepare(case, seed))
    st = prepare(case, seed)
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
    slot = st["slot"].long()
    pages = []
    for base, t in ((st["k"], res[1]), (st["v"], x[:, Hq + Hkv:])):
        full = base.double().view(-1, Hkv, d)
        full[slot] = t
        pages.append(full.view(base.shape))
    return res[0], pages[0], pages[1]


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
            K = st["k"].view(-1, Hkv, d)[flat, h].double()
            W = st["v"].view(-1, Hkv, d)[flat, h].double()
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
