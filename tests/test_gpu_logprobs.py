"""GPU parity of kda_token_logprobs with a 64-bit plain form: vocabularies from one
token to 2^24, rows of any alignment and stride, ties, masks that leave few tokens or
none, NaN and infinities, temperatures, rows on several CTAs, thousands of equal
logits; determinism, graphs and streams."""

import math

import pytest
import torch

import hybrid_linear_attention_delta_gb300 as kda

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DT = {"bf16": BF16, "f32": F32}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.lib()


def _call(logits, tokens, K, scale=1.0, ws=None, stream=None, want=("lp", "ent", "rank")):
    N = logits.shape[0]
    f = lambda *s: torch.full(s, 9.0, device="cuda")
    i = lambda *s: torch.full(s, 9, dtype=torch.int32, device="cuda")
    r = dict(lp=f(N), ent=f(N), rank=i(N), ids=i(N, K), top=f(N, K))
    ws = kda.paged_workspace_for() if ws is None else ws
    pick = {n: r[n] if n in want else None for n in ("lp", "ent", "rank")}
    kda.kda_token_logprobs(logits, tokens, pick["lp"], pick["ent"], pick["rank"],
                           r["ids"] if K else None, r["top"] if K else None, scale=scale,
                           workspace=ws, stream=stream)
    return r, ws


def _tolerance(V, d_max):
    """Absolute error of a log probability in 32-bit sums.  A thread adds up to V / 128
    terms in runs of 16, to a sum that is half of the last one on average; with the runs'
    own additions and the joins that is c half steps of the sum.  A term 2^d is off by 2^-22 and by the rounding of its exponent, |d| U
    ln 2; weighted with the term itself that is at most 0.6 U.  Then the logit's own
    distance to the largest is rounded a few times."""
    c = V / 256 / 16 + 40
    return c * U + 2.0 ** -21 + 6 * U * d_max


def _reference(logits, tokens, K, scale):
    """Row by row in 64 bits; places by a stable sort."""
    x = logits.double().cpu()
    N, V = x.shape
    out = dict(lp=[], ent=[], rank=[], ids=[], top=[])
    for n in range(N):
        y = x[n] * scale
        lse = torch.logsumexp(y, 0)
        lp = y - lse
        p = lp.exp()
        order = torch.sort(x[n], descending=True, stable=True).indices
        order = order[:int((x[n] > -math.inf).sum())][:K].tolist()
        out["ids"].append(order + [-1] * (K - len(order)))
        out["top"].append(lp[order].tolist() + [-math.inf] * (K - len(order)))
        out["ent"].append(float(-(p * torch.where(p > 0, lp, 0.0)).sum()))
        t = int(tokens[n]) if tokens is not None else -1
        if 0 <= t < V:
            out["lp"].append(float(lp[t]))
            out["rank"].append(int((x[n] > x[n, t]).sum() + (x[n, :t] == x[n, t]).sum()))
        else:
            out["lp"].append(0.0)
            out["rank"].append(-1)
    return out


def _check(logits, tokens, K, scale=1.0):
    r, ws = _call(logits, None if tokens is None else tokens.cuda(), K, scale,
                  want=("lp", "ent", "rank") if tokens is not None else ("ent",))
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    assert kda.kda_last_launch_count() == 1
    ref = _reference(logits, tokens, K, scale)
    V = logits.shape[1]
    finite = logits.float()[torch.isfinite(logits.float())]
    d_max = float(finite.max() - finite.min()) * scale + 20
    tol = _tolerance(V, d_max)
    N = logits.shape[0]
    assert r["ids"].tolist() == ref["ids"]
    if tokens is not None:
        assert r["rank"].tolist() == ref["rank"]
        names = ("lp", "ent", "top")
    else:
        names = ("ent", "top")
    for name in names:
        got = r[name].double().cpu().reshape(N, -1)
        want = torch.tensor(ref[name], dtype=torch.float64).reshape(N, -1)
        inf = want == -math.inf
        assert (got[inf] == -math.inf).all()
        # the entropy is a mean of |lp|: relative to itself too
        off = tol * (1 + (want.abs() if name == "ent" else 0))
        err = (got - want).abs()
        assert (err <= off)[~inf].all(), (name, float(err[~inf].max()), tol)
    return r


def _logits(N, V, kind, seed, std=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (std * torch.randn((N, V), generator=g, device="cuda")).to(DT[kind])


def _tokens(N, V, seed):
    return torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,K", [
    (1, 1, 1), (3, 2, 5), (2, 7, 7), (5, 8, 1), (4, 9, 3), (3, 31, 64), (1, 33, 0), (7, 1000, 20),
    (2, 4095, 64), (1, 4096, 64), (4, 50257, 5), (1, 131072, 64), (40, 65537, 20), (160, 9001, 2),
    (700, 1003, 1), (3, 200001, 33)])
def test_sizes(kind, N, V, K):
    _check(_logits(N, V, kind, V + N), _tokens(N, V, N), K)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.1, 1.7, 40.0])
def test_temperatures(kind, scale):
    _check(_logits(6, 5003, kind, 1), _tokens(6, 5003, 2), 8, scale)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_most_likely_tokens_as_given_tokens(kind):
    x = _logits(9, 30011, kind, 3)
    t = x.float().argmax(-1).int().cpu()
    r = _check(x, t, 4)
    if kind == "f32":
        assert torch.equal(r["lp"], r["top"][:, 0])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [2.0 ** -64, 1e-12, 0.25, 0.9, 1.0])
@pytest.mark.parametrize("V", [5, 3001])
def test_logits_further_apart_than_the_largest_float(kind, scale, V):
    """The largest logit and a token at the type's lowest value, whose difference is no
    float while its product with the scale may be one."""
    low, high = torch.finfo(DT[kind]).min, torch.finfo(DT[kind]).max
    x = _logits(4, V, kind, 6)
    x[:, 1] = low
    x[:, 3] = torch.tensor([high, high / 2, high / 64, 3e38], device="cuda").to(DT[kind])
    x[2, 4] = x[2, 3]
    K = 5
    r, ws = _call(x, torch.full((4,), 1, dtype=torch.int32, device="cuda"), K, scale)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    d = (x.double() - x.double().amax(1, keepdim=True)) * scale
    lp = (d - torch.logsumexp(d, 1, keepdim=True)).cpu()
    order = torch.sort(x.double(), descending=True, stable=True).indices[:, :K].cpu()
    assert torch.equal(r["ids"].cpu().long(), order)
    # (the scale, a difference, its product with it and the sum's logarithm are rounded once each)
    for got, want in ((r["lp"].cpu(), lp[:, 1]), (r["top"].cpu(), lp.gather(1, order))):
        inf = want < -torch.finfo(F32).max
        assert (got[inf] == -math.inf).all()
        assert ((got.double() - want).abs() <= 4 * U * want.abs() + 4 * U)[~inf].all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 3, 300])
def test_rows_of_any_stride_and_alignment(kind, N):
    """Rows that start on any element, with NaNs between them."""
    V, pad = 2003, 5
    full = torch.full((N * (V + pad) + 3,), float("nan"), dtype=DT[kind], device="cuda")
    for first in (0, 1, 3):
        x = full[first:first + N * (V + pad)].view(N, V + pad)[:, :V]
        x.copy_(_logits(N, V, kind, 5 + first))
        _check(x, _tokens(N, V, 6), 9)
        x.fill_(float("nan"))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [5, 4099, 131072])
def test_equal_logits(kind, V):
    """All equal (every place by its index), two values, and zeros of both signs."""
    N = 3
    x = torch.full((N, V), 1.5, dtype=DT[kind], device="cuda")
    t = torch.tensor([0, V - 1, V // 2], dtype=torch.int32)
    _check(x, t, 64)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = (torch.rand((N, V), generator=g, device="cuda") < 0.5).to(DT[kind])
    _check(x, t, 40)
    _check(-0.0 * x, t, 7)
    _check(-x * torch.where(x > 0, 0.0, 1.0).to(DT[kind]), t, 7)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("order", ["falling", "rising", "island", "strided", "block"])
def test_large_logits_in_one_place(kind, order):
    """The most likely tokens side by side, at the ends, or all in one thread's share."""
    V = 120000
    x = _logits(2, V, kind, 8, std=1.0)
    if order in ("falling", "rising"):
        x = torch.linspace(20, -20, V, device="cuda").expand(2, V).to(DT[kind]).contiguous()
        if order == "rising":
            x = x.flip(-1).contiguous()
    elif order == "island":
        x[:, 7777:7777 + 5000] += 30
    elif order == "strided":
        n = 8 if kind == "bf16" else 4
        at = torch.arange(V, device="cuda")
        x[:, (at // n) % 256 == 17] += 30
    else:
        x[:, -1500:] = (20 + torch.arange(1500, device="cuda") % 7).to(DT[kind])
    _check(x, torch.tensor([7800, V - 2], dtype=torch.int32), 64)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V,left", [(1000, 3), (50257, 1), (131072, 40), (131072, 30000)])
def test_masked_tokens(kind, V, left):
    """-inf nearly everywhere: fewer tokens than places, given tokens that are masked
    and that are not."""
    x = _logits(4, V, kind, 9)
    g = torch.Generator().manual_seed(left)
    hide = torch.ones((4, V), dtype=torch.bool)
    keep = torch.stack([torch.randperm(V, generator=g)[:left] for _ in range(4)])
    hide.scatter_(1, keep, False)
    x[hide.cuda()] = -math.inf
    gone = int(hide[2].nonzero()[5])
    _check(x, torch.tensor([int(keep[0, 0]), int(keep[1, -1]), gone, -1], dtype=torch.int32), 20)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [5, 1003, 50257])
@pytest.mark.parametrize("at", [-3e38, -1e30, -1e9, -9e5, 9e5, 1e9, 1e30, 3e38])
def test_logits_far_from_zero(kind, V, at):
    """Rows around a number of any size: the distribution is that of the differences, which
    are a few steps of the type there, at a scale that brings them to a few units."""
    g = torch.Generator().manual_seed(V)
    near = torch.tensor(at).to(DT[kind]).float()
    eps = 2.0 ** (torch.frexp(near).exponent.item() - (8 if kind == "bf16" else 24))
    x = (near.double() + eps * torch.randint(-9, 9, (3, V), generator=g)).to(DT[kind])
    t = _tokens(3, V, 3)
    scale = max(2.0 ** -64, 1 / eps)
    top = x.double().max(-1, keepdim=True).values
    ref = _reference(x.double() - top, t, 4, scale)
    r, ws = _call(x.cuda(), t.cuda(), 4, scale)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    tol = _tolerance(V, 20 + float((top - x.double().min()).max()) * scale)
    assert r["ids"].tolist() == ref["ids"] and r["rank"].tolist() == ref["rank"]
    for name, want in (("lp", ref["lp"]), ("ent", ref["ent"]), ("top", ref["top"])):
        want = torch.tensor(want, dtype=torch.float64)
        off = tol * (1 + (want.abs() if name == "ent" else 0))
        assert ((r[name].double().cpu() - want).abs() <= off).all(), name


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("low,scale", [(None, 2.0 ** -60), (None, 0.3), (None, 1.0), (None, 1e5),
                                       (-1e30, 1.0), (-1e9, 0.7), (-1e5, 10.0)])
@pytest.mark.parametrize("N,V,left", [(4, 6, 2), (4, 1000, 3), (2, 131072, 40), (400, 9001, 2000)])
def test_masks_of_low_values(kind, low, scale, N, V, left):
    """The type's lowest value, or another far below the others, in place of some -inf:
    what is left has the same distribution, the masked tokens come behind it; alone they are
    equal ones, also beside -inf."""
    x = _logits(N, V, kind, 11)
    x = (x.float() * min(1.0, 1 / scale)).to(DT[kind]) if scale > 1 else x
    low = float(torch.tensor(low).to(DT[kind])) if low else torch.finfo(DT[kind]).min
    g = torch.Generator().manual_seed(left)
    hide = torch.rand((N, V), generator=g) < 1 - left / V
    hide[:, V // 3] = False
    some = torch.tensor([low, -math.inf], dtype=DT[kind])[torch.randint(0, 2, (N, V), generator=g)]
    t = torch.full((N,), V // 3, dtype=torch.int32)
    t[1] = int(hide[1].nonzero()[0])
    hard = x.masked_fill(hide.cuda(), -math.inf)
    soft = torch.where(hide.cuda(), some.cuda(), x)
    ref = _reference(hard, t, 5, scale)
    r, ws = _call(soft, t.cuda(), 5, scale)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    seen = hard.float()[~hide.cuda()]
    # 2^-60: the lowest value is still 2^68 below the others when scaled
    tol = _tolerance(V, float(seen.max() - seen.min()) * scale + 20)
    rows = torch.arange(N) != 1
    assert ((r["lp"].cpu().double() - torch.tensor(ref["lp"]))[rows].abs() <= tol).all()
    # (a sum and two products of 32 bits)
    masked = float(soft[1, int(t[1])]) * scale - float(torch.logsumexp(hard[1].double() * scale, 0))
    assert r["lp"][1].item() == pytest.approx(masked, rel=1e-6) or masked < -3.4e38 and (
        r["lp"][1].item() == -math.inf)
    ent = torch.tensor(ref["ent"])
    assert ((r["ent"].cpu().double() - ent).abs() <= tol * (1 + ent.abs())).all()
    order = torch.sort(soft.double().cpu(), descending=True, stable=True)
    ids = torch.where(order.values > -math.inf, order.indices, -1)[:, :5]
    assert r["ids"].cpu().tolist() == ids.tolist()
    assert r["rank"][0] == ref["rank"][0]
    # nothing but masks: the lowest values share the row
    some[:, 0] = low
    r, ws = _call(some.cuda(), t.cuda(), 5, scale)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    n = (some > -math.inf).sum(-1).double()
    tol = _tolerance(V, 20)
    assert ((r["ent"].cpu().double() - n.log()).abs() <= tol * (1 + n.log())).all()
    assert ((r["top"][:, 0].cpu().double() + n.log()).abs() <= tol).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [6, 1000, 131072])
@pytest.mark.parametrize("N", [3, 400])
def test_rows_without_a_distribution(kind, V, N):
    """Nothing left, NaN, +inf: said with an error bit, the other rows as ever."""
    x = _logits(N, V, kind, 4)
    t = _tokens(N, V, 1)
    clean, _ = _call(x, t.cuda(), 5)
    x[1] = -math.inf
    r, ws = _call(x, t.cuda(), 5)
    assert kda.kda_device_status(ws) == (kda.KDA_ERR_DEVICE_CHECK, 4096)
    assert r["lp"][1] == -math.inf and r["ent"][1] == 0
    assert r["ids"][1].tolist() == [-1] * 5 and (r["top"][1] == -math.inf).all()
    rest = torch.arange(N, device="cuda") != 1
    for n in clean:
        assert torch.equal(r[n][rest], clean[n][rest])
    for bad, at in ((math.nan, 0), (math.inf, V - 1), (math.nan, V // 2)):
        x[1] = 1.0
        x[1, at] = bad
        r, ws = _call(x, t.cuda(), 5)
        assert kda.kda_device_status(ws) == (kda.KDA_ERR_DEVICE_CHECK, 16384)
        assert r["lp"][1].isnan() and r["ent"][1].isnan() and r["rank"][1] == -1
        assert r["ids"][1].tolist() == [-1] * 5 and r["top"][1].isnan().all()
        for n in clean:
            assert torch.equal(r[n][rest], clean[n][rest])


def test_tokens_that_are_none():
    x = _logits(3, 500, "f32", 2)
    r, ws = _call(x, torch.tensor([-1, 500, -9], dtype=torch.int32, device="cuda"), 2)
    assert kda.kda_device_status(ws) == (kda.KDA_ERR_DEVICE_CHECK, 2048)
    assert r["lp"].tolist() == [0, 0, 0] and r["rank"].tolist() == [-1] * 3


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_outputs_that_are_not_asked_for(kind):
    x, t = _logits(5, 3001, kind, 2), _tokens(5, 3001, 3)
    every, _ = _call(x, t.cuda(), 6)
    for want in (("lp",), ("ent",), ("rank",), ()):
        r, _ = _call(x, t.cuda(), 6, want=want)
        for n in ("lp", "ent", "rank"):
            assert torch.equal(r[n], every[n]) if n in want else (r[n] == 9).all()
        assert torch.equal(r["ids"], every["ids"]) and torch.equal(r["top"], every["top"])
    _check(x, None, 6)
    r, _ = _call(x, t.cuda(), 0)
    assert torch.equal(r["lp"], every["lp"])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_the_largest_vocabulary(kind):
    """2^24 tokens: a thread's segments are longer, its sums too."""
    V = 1 << 24
    x = _logits(2, V, kind, 6)
    _check(x, _tokens(2, V, 6), 64)


def test_offsets_beyond_32_bits():
    """More than 2^31 logits; the last rows against rows of their own."""
    V, N = 131072, (1 << 31) // 131072 + 9
    x = torch.zeros((N, V), dtype=BF16, device="cuda")
    x[-4:] = _logits(4, V, "bf16", 3)
    t = _tokens(N, V, 2)
    r, ws = _call(x, t.cuda(), 3)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    ref = _reference(x[-4:], t[-4:], 3, 1.0)
    assert r["ids"][-4:].tolist() == ref["ids"] and r["rank"][-4:].tolist() == ref["rank"]
    assert (r["lp"][-4:].cpu().double() - torch.tensor(ref["lp"])).abs().max() <= _tolerance(V, 60)
    assert (r["ids"][:-4] == torch.arange(3, device="cuda")).all()
    assert (r["ent"][:-4] - math.log(V)).abs().max() <= _tolerance(V, 60) * 13


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_near_certain_rows(kind):
    """One token has nearly all the mass: an entropy near 0 that is not negative."""
    x = _logits(4, 50000, kind, 7, std=1.0)
    x[:, 123] = torch.tensor([20.0, 30.0, 60.0, 200.0], device="cuda").to(DT[kind])
    r = _check(x, torch.full((4,), 123, dtype=torch.int32), 3)
    assert (r["ent"] >= 0).all() and (r["lp"] <= 0).all()


def test_repeats_graphs_and_streams():
    """The same bits at every call, in a replayed graph, and on two streams at once."""
    cases = [(_logits(5, 50257, "bf16", 1), _tokens(5, 50257, 1).cuda()),
             (_logits(300, 9001, "f32", 2), _tokens(300, 9001, 2).cuda())]
    firsts = [_call(x, t, 20)[0] for x, t in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        rs = [_call(x, t, 20, stream=s)[0] for (x, t), s in zip(cases, streams)]
        torch.cuda.synchronize()
        for r, first in zip(rs, firsts):
            for n in r:
                assert torch.equal(r[n], first[n])
    ws = kda.paged_workspace_for()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rs = [_call(x, t, 20, ws=ws)[0] for x, t in cases]
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for r, first in zip(rs, firsts):
            for n in r:
                assert torch.equal(r[n], first[n])
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
