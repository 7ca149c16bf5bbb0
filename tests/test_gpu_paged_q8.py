"""GPU parity of kda_paged_append_q8 and kda_paged_attn_q8 with 64-bit plain forms:
lengths from one token to long chunks, odd lengths and tile borders, every page and
group size, rows that see nothing, scales far apart, blocks without a scale, poisoned
memory around the keys; blocks that grow; determinism, graphs and streams."""

import pytest
import torch

import hybrid_linear_attention_delta_gb300 as kda
from kda_cases import TOL
from paged_cases import BF16, DT, F32, append_reference, half_step
from q8_cases import BLOCK, E4M3, NAN8, Q8AttnCase, append_blocks, rounded, scale_for, spread

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.lib()


# ------------------------------------------------------------------- attention

def _call(t, out, ws, **kw):
    kda.kda_paged_attn_q8(t["q"], t["k8"], t["v8"], t["k_scales"], t["v_scales"], t["table"],
                          t["cu"], t["kv"], out, workspace=ws, **kw)


def _run(case, causal=True, scale=None, dev=None, ws=None, out=None):
    t = dev or case.cuda()
    if out is None:
        out = torch.full_like(t["q"], case.MARK)
    if ws is None:
        ws = kda.paged_workspace_for(t["q"].shape[0], case.Hq, case.Hkv, case.d)
    _call(t, out, ws, scale=scale, causal=causal)
    return out, ws


def _near(case, out, causal=True, scale=None, rows=slice(None)):
    ref, size, top = case.reference(causal, scale)
    got = out.double().cpu()
    assert torch.isfinite(got[rows]).all()
    err = (got - ref)[rows].abs()
    over = err > case.bound(ref, size, top)[rows]
    assert not over.any(), (float(err.max()), int(over.sum()), over.nonzero()[:4].tolist())
    return got, ref


def _check(case, causal=True, scale=None, norm_bar=True):
    out, ws = _run(case, causal, scale)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    assert kda.kda_last_launch_count() == 1
    used = int(case.cu[-1])
    got, ref = _near(case, out, causal, scale, slice(0, used))
    name = "bf16" if case.dtype == BF16 else "f32"
    if norm_bar and used and float(ref.norm()) > 0:
        assert float((got - ref)[:used].norm() / ref.norm()) <= TOL[name]
    assert (out[used:] == case.MARK).all()              # rows behind the last request
    assert int(ws[256:256 + 8 * 304].sum()) == 0        # counters are left as they were found
    return out


LENGTHS = [
    ([1], [1]), ([1], [777]), ([1, 1, 1], [127, 128, 129]), ([5], [5]), ([64], [200]),
    ([130], [130]), ([1, 0, 7, 33], [40, 0, 7, 300]), ([200, 3], [200, 1000]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,total", LENGTHS)
def test_lengths(dtype, d, new, total):
    _check(Q8AttnCase(new, total, Hq=8, Hkv=2, d=d, page=16, dtype=dtype, seed=len(new), pad=3))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(dtype, page):
    for d in (64, 128):
        _check(Q8AttnCase([70, 1, 9], [333, 257, 256], Hq=4, Hkv=2, d=d, page=page, dtype=dtype,
                          seed=page))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (3, 1), (10, 2), (7, 1), (16, 1), (24, 1),
                                    (64, 1), (33, 3)])
def test_groups(dtype, Hq, Hkv):
    """Groups that fill a tile of rows and groups that leave some of it empty."""
    _check(Q8AttnCase([43, 1, 150], [300, 200, 151], Hq=Hq, Hkv=Hkv, d=64, page=32, dtype=dtype,
                      seed=Hq))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_nothing(dtype, causal, d):
    """No keys at all, and more new tokens than keys: their rows are zeros."""
    case = Q8AttnCase([4, 9, 1, 300], [0, 3, 50, 20], Hq=6, Hkv=2, d=d, page=16, dtype=dtype)
    out = _check(case, causal)
    assert (out[:4] == 0).all()
    if causal:
        assert (out[4:10] == 0).all() and (out[10:13] != 0).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_not_causal_and_scale(dtype, d):
    case = Q8AttnCase([40, 1], [500, 77], Hq=4, Hkv=1, d=d, page=64, dtype=dtype)
    _check(case, causal=False)
    for scale in (0.02, 0.0, -0.05):
        _check(case, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 128), (8, 1, 128), (16, 8, 64)])
def test_long_context_is_split_and_joined(dtype, Hq, Hkv, d):
    """Few rows over many keys: pieces on every SM, joined in order."""
    case = Q8AttnCase([1], [20011], Hq=Hq, Hkv=Hkv, d=d, page=16, dtype=dtype, seed=5)
    a = _check(case)
    for _ in range(3):
        assert torch.equal(a, _run(case)[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,new", [(3, 1), (4, 1), (5, 1), (8, 2), (17, 1), (64, 2), (7, 30)])
def test_pieces_are_joined_whatever_the_rows(dtype, d, G, new):
    _check(Q8AttnCase([new, 1], [9001, 130], Hq=2 * G, Hkv=2, d=d, page=64, dtype=dtype, seed=G))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [2.0 ** -60, 1.0, 2.0 ** 60])
def test_sizes_of_queries(dtype, size):
    """Queries of any magnitude, and rows whose channels are far apart."""
    case = Q8AttnCase([50, 1], [300, 77], Hq=4, Hkv=2, d=128, page=16, dtype=dtype, seed=2)
    case.q = (case.q.double() * size).to(case.dtype)
    case.q[::3, :, 5] *= 64
    case.q[1::3] = 0
    _check(case, scale=0.05 / size)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_large_scores(dtype, d):
    """Scores that differ by hundreds: a few keys carry all the weight."""
    case = Q8AttnCase([50, 1], [700, 2900], Hq=4, Hkv=2, d=d, page=16, dtype=dtype, seed=9,
                      scale_q=40.0)
    _check(case, norm_bar=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,new,total", [
    (2, 1, [130], [1500]),            # two tiles of rows
    (4, 2, [300, 1, 0, 9], [900, 2900, 5, 640]),  # both forms of item, ragged ends
    (8, 1, [1], [20011]),             # one item over many CTAs
    (64, 1, [5], [6000]),             # both tiles of rows over many CTAs
])
@pytest.mark.parametrize("kind", ["rising", "falling", "steps"])
def test_references_move(d, Hq, Hkv, new, total, kind):
    """Scores that pass a row's reference from tile to tile, or fall."""
    case = Q8AttnCase(new, total, Hq=Hq, Hkv=Hkv, d=d, page=16, dtype="bf16", seed=d + Hq)
    k = torch.nan_to_num(case.k)
    for b, t in enumerate(total):
        at = torch.arange(t, dtype=torch.float64)
        ramp = {"rising": -40 + 80 * at / t, "falling": 40 - 80 * at / t,
                "steps": 10.0 * (at // 200)}[kind]
        ids = case.table[b, :-(-t // 16)].long()
        rows = k[ids].reshape(-1, Hkv, d)
        rows[:t, :, 0] = ramp[:, None]
        k[ids] = rows.reshape(-1, 16, Hkv, d)
    case.set_values("k", k, 4.0)      # up to 1000 of 1792
    rows = torch.arange(case.q.shape[0])[:, None] % 3
    case.q[..., 0] = (torch.tensor([6.0, 0.5, 20.0])[rows]).to(BF16)
    _check(case, norm_bar=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("powers", [(-50, -49), (-50, 40), (48, 49), (-3, 12)])
def test_scales_of_values_far_apart(dtype, d, powers):
    """Values whose scales differ by up to 2^90 from block to block, and scales at the
    ends of their range."""
    case = Q8AttnCase([130, 1, 3], [700, 900, 2000], Hq=4, Hkv=2, d=d, page=32, dtype=dtype,
                      seed=d)
    g = torch.Generator().manual_seed(4)
    power = torch.randint(powers[0], powers[1] + 1, case.v_scales.shape, generator=g)
    case.v_scales = torch.where(torch.isnan(case.v_scales), case.v_scales, torch.exp2(power.float()))
    case.v = case.v8.double() * spread(case.v_scales)
    _check(case)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales_of_keys_far_apart(dtype):
    case = Q8AttnCase([40, 1], [700, 900], Hq=4, Hkv=2, d=128, page=16, dtype=dtype, seed=3,
                      powers=(-30, -5))
    _check(case)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("which", ["k_scales", "v_scales"])
@pytest.mark.parametrize("bad", [float("nan"), 0.0, -1.0, float("inf"), 2.0 ** -51, 2.0 ** 51])
def test_blocks_without_a_scale_are_left_out(dtype, which, bad):
    """Keys 16..31 of one head of request 0 and all of request 1's count for nothing."""
    new, total = [70, 1, 9], [300, 16, 200]
    case = Q8AttnCase(new, total, Hq=4, Hkv=2, d=64, page=16, dtype=dtype, seed=6)
    getattr(case, which)[case.table[0, 1].long(), 0, 1] = bad
    getattr(case, which)[case.table[1, 0].long(), 0, :] = bad
    out, ws = _run(case)
    assert kda.kda_device_status(ws) == (kda.KDA_ERR_DEVICE_CHECK, 8192)
    whole = Q8AttnCase(new, total, Hq=4, Hkv=2, d=64, page=16, dtype=dtype, seed=6)
    ref, size, top = whole.reference()
    c = whole.d ** -0.5
    ids = whole.table[0, :-(-300 // 16)].long()
    keep = torch.ones(300, dtype=torch.bool)
    keep[16:32] = False
    K, W = (x[ids].flatten(0, 1)[:300, 1] for x in (whole.k, whole.v))
    for h in (2, 3):
        s = c * whole.q[:70, h].double() @ K.T
        s.masked_fill_(torch.arange(300)[None] > 230 + torch.arange(70)[:, None], -float("inf"))
        w = torch.softmax(s.masked_fill(~keep, -float("inf")), -1)
        ref[:70, h] = w @ torch.nan_to_num(W)
        size[:70, h] = w @ torch.nan_to_num(W).abs()
    ref[70:71] = size[70:71] = 0
    assert ((out.double().cpu() - ref).abs() <= whole.bound(ref, size, top)).all()


def test_mixed_batch_of_many_requests():
    g = torch.Generator().manual_seed(11)
    new = torch.randint(0, 60, (90,), generator=g).tolist()
    total = [n + c for n, c in zip(new, torch.randint(0, 400, (90,), generator=g).tolist())]
    _check(Q8AttnCase(new, total, Hq=6, Hkv=2, d=128, page=16, dtype="bf16", seed=12, pad=17))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 4, 16])
@pytest.mark.parametrize("causal", [True, False])
def test_a_chunk_in_a_padded_batch(d, G, causal):
    """Few rows a request on average, nearly all of them one request's: many items of it."""
    new = [0, 0, 150, 0, 1] + [0] * (12 * G + 100) + [1, 2, 0]
    total = [9, 0, 700, 0, 3000] + [0] * (12 * G + 100) + [40, 2, 7]
    _check(Q8AttnCase(new, total, Hq=3 * G, Hkv=3, d=d, page=32, dtype="bf16", seed=G, pad=9),
           causal)


@pytest.mark.parametrize("d,G", [(64, 1), (128, 2), (64, 16), (128, 24)])
@pytest.mark.parametrize("Hkv", [2, 5, 8])
def test_stretches_that_cross_heads(d, G, Hkv):
    """More items than CTAs, of a request or of many: a CTA goes from the last request of
    one head to the first of the next, past empty ones at either end."""
    g = torch.Generator().manual_seed(Hkv + d)
    new = [0, 0] + torch.randint(0, 4, (90,), generator=g).tolist() + [0, 0, 0]
    total = [n + c for n, c in zip(new, torch.randint(0, 300, (95,), generator=g).tolist())]
    _check(Q8AttnCase(new, total, Hq=G * Hkv, Hkv=Hkv, d=d, page=16, dtype="bf16", seed=Hkv))
    _check(Q8AttnCase([3], [9], Hq=G * Hkv, Hkv=Hkv, d=d, page=16, dtype="bf16", seed=Hkv))


@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_that_see_nothing(d):
    """As test_rows_that_see_nothing, with no more rows than the small products take."""
    case = Q8AttnCase([4, 2, 1, 6], [0, 1, 50, 3], Hq=2, Hkv=2, d=d, page=16, dtype="bf16", seed=4)
    out = _check(case)
    assert (out[:5] == 0).all() and (out[7:10] == 0).all()
    assert (out[5:7] != 0).any() and (out[10:13] != 0).any()
    assert (_check(case, causal=False)[4:] != 0).any()


@pytest.mark.parametrize("d", [64, 128])
def test_chunk_against_a_long_prefix(d):
    _check(Q8AttnCase([519], [4100], Hq=8, Hkv=2, d=d, page=128, dtype="bf16", seed=21))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_short_requests(dtype):
    g = torch.Generator().manual_seed(31)
    new = torch.randint(0, 3, (1500,), generator=g).tolist()
    total = [n + c for n, c in zip(new, torch.randint(0, 40, (1500,), generator=g).tolist())]
    _check(Q8AttnCase(new, total, Hq=2, Hkv=1, d=64, page=16, dtype=dtype, seed=32, pad=5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_beyond_32_bit_offsets(dtype):
    """A pool of more than 2^32 bytes, with the request's pages at its end."""
    Hkv, d, page = 8, 128, 256
    case = Q8AttnCase([3, 1], [600, 90], Hq=8, Hkv=Hkv, d=d, page=page, dtype=dtype, seed=4)
    t = case.cuda()
    n_small = case.k8.shape[0]
    n_pages = (1 << 32) // (page * Hkv * d) + 40
    for n in ("k8", "v8"):
        big = torch.zeros((n_pages, page, Hkv, d), dtype=E4M3, device="cuda")
        big.view(torch.uint8)[n_pages - n_small:] = t[n].view(torch.uint8)
        t[n] = big
    for n in ("k_scales", "v_scales"):
        big = torch.zeros((n_pages, page // BLOCK, Hkv), device="cuda")
        big[n_pages - n_small:] = t[n]
        t[n] = big
    t["table"] = t["table"] + (n_pages - n_small)
    out, ws = _run(case, dev=t)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    _near(case, out)


@pytest.mark.parametrize("d,Hkv,G,B,T,lg", [
    (128, 4, 4, 1, 1280, 21), (64, 4, 3, 1, 1000, 21), (128, 2, 4, 20, 1, 23), (64, 2, 8, 1, 2, 24)])
def test_sums_over_millions_of_keys(d, Hkv, G, B, T, lg):
    """Values of one sign over the same sixteen pages again and again."""
    g = torch.Generator(device="cuda").manual_seed(lg + d)
    page, n_pages, kv = 256, 16, 1 << lg
    k8 = (64 * torch.randn((n_pages, page, Hkv, d), generator=g, device="cuda")).clamp(-448, 448).to(E4M3)
    v8 = (32 * torch.rand((n_pages, page, Hkv, d), generator=g, device="cuda") + 16).to(E4M3)
    scales = torch.full((n_pages, page // BLOCK, Hkv), 2.0 ** -6, device="cuda")
    q = torch.randn((B * T, Hkv * G, d), generator=g, device="cuda").bfloat16()
    table = (torch.arange(1 << lg - 8, device="cuda") % n_pages).int().repeat(B, 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    t = dict(q=q, k8=k8, v8=v8, k_scales=scales, v_scales=scales, table=table,
             cu=i32([T * b for b in range(B + 1)]), kv=i32([kv] * B))
    ws = kda.paged_workspace_for(B * T, Hkv * G, Hkv, d)
    outs = [torch.zeros_like(q) for _ in range(2)]
    for out in outs:
        _call(t, out, ws, causal=False)
        assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    assert torch.equal(*outs)
    ref = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for h in range(Hkv * G):
        K, W = (x[:, :, h // G].flatten(0, 1).double() * 2.0 ** -6 for x in (k8, v8))
        ref[:, h] = torch.softmax(q[:, h].double() @ K.T * d ** -0.5, -1) @ W
    # as for the 16-bit cache: weights and outputs are rounded once each (at most 2^-8),
    # and a run of 2^17 keys loses at most 2^-10 of its sum
    err = outs[0].double() - ref
    assert (err.abs() <= ref.abs() * (2 * 2.0 ** -8 * 1.01 + 2.0 ** -10)).all()
    assert float(err.norm() / ref.norm()) <= TOL["bf16"]


@pytest.mark.parametrize("d", [64, 128])
def test_sums_of_few_rows_over_millions_of_keys(d):
    """A token a request over some 2^23 keys, the same sixteen pages again and again: pieces
    of more than 2^19 keys, whose sums are put aside on the way, and lengths that end each of
    a CTA's warps at another step."""
    g = torch.Generator(device="cuda").manual_seed(d)
    page, n_pages, Hkv, G, B = 256, 16, 2, 4, 20
    period = page * n_pages
    kv = [(1 << 23) + 16 * 5 * b + b % 7 for b in range(B)]
    k8 = (64 * torch.randn((n_pages, page, Hkv, d), generator=g, device="cuda")).clamp(-448, 448).to(E4M3)
    v8 = (32 * torch.rand((n_pages, page, Hkv, d), generator=g, device="cuda") + 16).to(E4M3)
    scales = torch.full((n_pages, page // BLOCK, Hkv), 2.0 ** -6, device="cuda")
    q = torch.randn((B, Hkv * G, d), generator=g, device="cuda").bfloat16()
    table = (torch.arange(-(-max(kv) // page), device="cuda") % n_pages).int().repeat(B, 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    t = dict(q=q, k8=k8, v8=v8, k_scales=scales, v_scales=scales, table=table,
             cu=i32(list(range(B + 1))), kv=i32(kv))
    ws = kda.paged_workspace_for(B, Hkv * G, Hkv, d)
    outs = [torch.zeros_like(q) for _ in range(2)]
    for out in outs:
        _call(t, out, ws)
        assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    assert torch.equal(*outs)
    # how often a request sees each of the keys
    at = torch.arange(period, device="cuda")
    often = torch.stack([(n // period + (at < n % period)).double() for n in kv])
    ref = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for h in range(Hkv * G):
        K, W = (x[:, :, h // G].flatten(0, 1).double() * 2.0 ** -6 for x in (k8, v8))
        s = q[:, h].double() @ K.T * d ** -0.5
        w = often * torch.exp(s - s.amax(-1, keepdim=True))
        ref[:, h] = w @ W / w.sum(-1, keepdim=True)
    # Weights (2^-11) and outputs (2^-8) are rounded once; a run of 8192 additions, each off
    # by at most 2^-23 (products) or 2^-24 (weights) of its sum.
    err = (outs[0].double() - ref).abs()
    assert (err <= ref.abs() * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -10 + 2.0 ** -11) * 1.01).all()
    assert float(err.norm() / ref.norm()) <= TOL["bf16"]


def test_captured_graphs_share_a_workspace_and_follow_the_lengths():
    cases = [Q8AttnCase([1, 1], [900, 300], Hq=8, Hkv=2, d=128, page=16, dtype="bf16", seed=1),
             Q8AttnCase([40, 9], [140, 2000], Hq=8, Hkv=2, d=128, page=32, dtype="bf16", seed=2)]
    ws = kda.paged_workspace_for(64, 8, 2, 128)
    devs = [c.cuda() for c in cases]
    outs = [torch.zeros_like(t["q"]) for t in devs]
    for c, t, o in zip(cases, devs, outs):
        _run(c, dev=t, ws=ws, out=o)
    torch.cuda.synchronize()
    graphs = []
    for c, t, o in zip(cases, devs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _run(c, dev=t, ws=ws, out=o)
        graphs.append(g)
    for _ in range(3):
        for g, o in zip(graphs, outs):
            o.zero_()
            g.replay()
    for c, o in zip(cases, outs):
        _near(c, o)
    # shorter requests in the captured call
    cases[0].total = [500, 17]
    devs[0]["kv"].copy_(torch.tensor([500, 17], dtype=torch.int32))
    graphs[0].replay()
    _near(cases[0], outs[0])
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)


def test_two_calls_at_once_on_streams_of_their_own():
    cases = [Q8AttnCase([1, 40], [3000, 700], Hq=8, Hkv=2, d=d, page=16, dtype="bf16", seed=d)
             for d in (64, 128)]
    devs = [c.cuda() for c in cases]
    outs = [torch.zeros_like(t["q"]) for t in devs]
    wss = [kda.paged_workspace_for(41, 8, 2, c.d) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for t, o, ws, s in zip(devs, outs, wss, streams):
            _call(t, o, ws, stream=s)
    torch.cuda.synchronize()
    for c, o, ws in zip(cases, outs, wss):
        _near(c, o)
        assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,d", [(8, 128), (3, 64)])
def test_out_over_q(dtype, G, d):
    case = Q8AttnCase([1, 90, 0, 301, 2], [9000, 700, 5, 301, 4000], Hq=2 * G, Hkv=2, d=d, page=32,
                      dtype=dtype, seed=G)
    apart, _ = _run(case)
    t = case.cuda()
    ws = kda.paged_workspace_for(t["q"].shape[0], 2 * G, 2, d)
    _call(t, t["q"], ws)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    assert torch.equal(t["q"], apart)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_nan_stays_in_its_row(dtype):
    """A query that holds a NaN gives NaNs, and nothing else does."""
    case = Q8AttnCase([70], [300], Hq=2, Hkv=1, d=64, page=16, dtype=dtype, seed=8)
    clean, _ = _run(case)
    case.q[33, 1, 5] = float("nan")
    out, _ = _run(case)
    assert out[33, 1].isnan().all()
    keep = torch.ones(70, 2, dtype=torch.bool)
    keep[33, 1] = False
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_key_counts_for_the_rows_that_see_it(dtype, d):
    """A cached NaN among the keys gives NaNs in the rows that see it, and in no
    others' results; behind the request's last key nothing counts."""
    case = Q8AttnCase([70], [300], Hq=2, Hkv=1, d=d, page=16, dtype=dtype, seed=8)
    clean, _ = _run(case)
    case.k8.view(torch.uint8)[int(case.table[0, 270 // 16]), 270 % 16, 0, 3] = NAN8
    out, _ = _run(case)
    assert out[40:].isnan().all()               # row 40 sits at position 270
    assert torch.equal(out[:40], clean[:40])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_lengths_tables_and_pages(dtype):
    """Inputs that the device checks refuse: an error bit, and nothing else."""
    mk = lambda: Q8AttnCase([3, 5], [40, 60], Hq=4, Hkv=2, d=64, page=16, dtype=dtype)
    for cu in ([0, 9, 8], [1, 3, 8], [0, 3, 9]):
        case = mk()
        case.cu = torch.tensor(cu, dtype=torch.int32)
        out, ws = _run(case)
        assert kda.kda_device_status(ws) == (kda.KDA_ERR_DEVICE_CHECK, 4)
        assert (out == case.MARK).all()
    for bad in (-1, 65):     # negative; beyond the table's four pages
        case = mk()
        ref, size, top = case.reference()
        case.kv[1] = bad
        out, ws = _run(case)
        assert kda.kda_device_status(ws) == (kda.KDA_ERR_DEVICE_CHECK, 128)
        assert (out[3:] == case.MARK).all()
        assert ((out.double().cpu() - ref)[:3].abs() <= case.bound(ref, size, top)[:3]).all()
    for page in (-5, 1 << 20):   # reads as zeros: keys and values 16..31 of request 0
        case = mk()
        good = int(case.table[0, 1])
        t = case.cuda()
        t["table"][0, 1] = page
        case.k[good], case.v[good] = 0, 0
        out, ws = _run(case, dev=t)
        assert kda.kda_device_status(ws) == (kda.KDA_ERR_DEVICE_CHECK, 512)
        _near(case, out)


# ---------------------------------------------------------------------- append

class Cache:
    """An 8-bit cache with something in every slot."""

    def __init__(self, n_pages, page, Hkv, d, g, power=(-8, -4)):
        self.page, self.n_slots = page, n_pages * page
        self.pages, self.scales = [], []
        for _ in range(2):
            x = (60 * torch.randn((n_pages, page, Hkv, d), generator=g)).clamp(-448, 448)
            self.pages.append(x.to(E4M3))
            e = torch.randint(*power, (n_pages, page // BLOCK, Hkv), generator=g)
            self.scales.append(torch.exp2(e.float()))


def _append(cache, qkv, slots, Hq, Hkv, *, q_norm=None, k_norm=None, rope=None, positions=None,
            mode="half", eps=1e-6, stream=None):
    dev = lambda t: None if t is None else t.cuda()
    T, _, d = qkv.shape
    q = torch.full((T, Hq, d), 7.0, dtype=qkv.dtype, device="cuda")
    pages, scales = [dev(x) for x in cache.pages], [dev(x) for x in cache.scales]
    ws = kda.paged_workspace_for()
    args = (dev(qkv), dev(q_norm), dev(k_norm), dev(rope), dev(positions), dev(slots.int()), q,
            *pages, *scales)
    kda.kda_paged_append_q8(*args, rope_mode=mode, norm_eps=eps, workspace=ws, stream=stream)
    status = kda.kda_device_status(ws)
    assert kda.kda_last_launch_count() in (0, 1)
    return q.cpu(), [x.cpu() for x in pages], [x.cpu() for x in scales], status


def _check_append(cache, qkv, slots, Hq, Hkv, kind, **kw):
    """Values that reach the cache unrounded (v; k without norm and rotation) must be
    the exact results.  Others are off by the fp32 error e of norm and rotation, then
    rounded: a value by at most max(2^-4 |x|, 2^-10 s) + e, a scale is that of a largest
    value between amax - e and amax + e."""
    q, pages, scales, status = _append(cache, qkv, slots, Hq, Hkv, **kw)
    assert status == (kda.KDA_OK, 0)
    T, _, d = qkv.shape
    pos = kw.get("positions")
    (rq, sq), (rk, sk), rv = append_reference(
        qkv, kw.get("q_norm"), kw.get("k_norm"), kw.get("rope"), pos if pos is not None else
        torch.zeros(T, dtype=torch.int32), Hq, Hkv, kw.get("mode", "half"), kw.get("eps", 1e-6))
    u = half_step(F32)
    real = slots >= 0
    e_rel = (d + 16) * u if kw.get("k_norm") is not None or kw.get("q_norm") is not None else 8 * u
    off = half_step(DT[kind]) * rq.abs() * 1.01 + e_rel * sq * 2 + 1e-30
    assert ((q.double() - rq).abs() <= off)[real].all()
    assert (q[~real] == 7.0).all()
    changed = kw.get("k_norm") is not None or kw.get("rope") is not None
    for i, (x, e) in enumerate(((rk, e_rel * sk * 2 if changed else torch.zeros_like(sk)),
                                (rv, torch.zeros_like(rv)))):
        old_p, old_s = cache.pages[i].double().view(-1, BLOCK, Hkv, d), cache.scales[i].double().view(-1, Hkv)
        got_p, got_s = pages[i].double().view(-1, BLOCK, Hkv, d), scales[i].double().view(-1, Hkv)
        new, comes, first = append_blocks(x, slots, cache.pages[i], cache.scales[i])
        err = append_blocks(e, slots, cache.pages[i], cache.scales[i])[0]
        hit = comes.any(1)
        held = torch.where((first == 0)[:, None], 0.0, old_s)
        top = torch.nan_to_num(new.abs() + err, nan=0.0).amax((1, 3))
        low = torch.nan_to_num(new.abs() - err, nan=0.0).amax((1, 3))
        s_hi, s_lo = (torch.maximum(held, scale_for(y)) for y in (top, low))
        assert ((got_s <= s_hi) & (got_s >= s_lo))[hit].all()
        assert torch.equal(got_s[~hit], old_s[~hit])
        s = got_s[:, None, :, None]
        # what was there before: rounded again where the scale grew
        before = (torch.arange(BLOCK)[None] < first[:, None]) & hit[:, None]
        ratio = (old_s[:, None, :, None] / s)
        again = torch.where(ratio == 1, old_p, rounded(old_p * ratio))
        assert torch.equal(got_p[before], again.expand_as(old_p)[before])
        # slots that nothing is written to
        rest = ~before & ~comes
        assert torch.equal(got_p[rest], old_p[rest])
        # the new ones
        if not (e != 0).any():
            want = rounded(new / s)
            assert torch.equal(got_p[comes], want[comes])
        got, x, e = (got_p * s)[comes], new[comes], err[comes]
        step = torch.maximum(2.0 ** -4 * (x.abs() + e), 2.0 ** -10 * s.expand_as(new)[comes])
        assert ((got - x).abs() <= step * (1 + 1e-9) + e).all()
    return q, pages, scales


def _runs(lengths, page, g, n_pages):
    """Slots of requests whose new tokens start anywhere in a page."""
    order = torch.randperm(n_pages, generator=g).tolist()
    slots = []
    for n in lengths:
        off = int(torch.randint(0, page, (1,), generator=g))
        for i in range(n):
            if i == 0 or (off + i) % page == 0:
                p = order.pop()
            slots.append(p * page + (off + i) % page)
    return torch.tensor(slots)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d,rots", [(64, (0, 16, 32, 64)), (128, (0, 16, 48, 64, 128))])
@pytest.mark.parametrize("mode", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [True, False])
def test_append_rotations_and_norms(kind, d, rots, mode, norm):
    g = torch.Generator().manual_seed(d)
    Hq, Hkv, page = 6, 2, 32
    for rot in rots:
        slots = _runs([1, 40, 16, 3, 1, 1], page, g, 30)
        T = len(slots)
        qkv = (torch.randn((T, Hq + 2 * Hkv, d), generator=g)
               * torch.exp2(torch.randn((T, 1, 1), generator=g))).to(DT[kind])
        kw = dict(mode=mode)
        if norm:
            kw.update(q_norm=1 + 0.1 * torch.randn(d, generator=g), k_norm=1 + 0.1 * torch.randn(d, generator=g))
        if rot:
            kw.update(rope=kda.rope_table(500, rot, device="cpu"),
                      positions=torch.randint(0, 500, (T,), generator=g).int())
        _check_append(Cache(30, page, Hkv, d, g), qkv, slots, Hq, Hkv, kind, **kw)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,Hq,Hkv,d,page", [
    ([1], 1, 1, 64, 16), ([1], 32, 8, 128, 64), ([2, 1], 5, 1, 128, 16), ([15], 4, 4, 64, 16),
    ([16], 3, 3, 128, 16), ([17], 7, 1, 64, 32), ([31, 33], 8, 2, 128, 16), ([1] * 70, 4, 2, 64, 32),
    ([600], 4, 2, 128, 128), ([1] * 400, 2, 1, 64, 16), ([1500, 7, 900], 2, 2, 64, 256)])
def test_append_shapes(kind, lengths, Hq, Hkv, d, page):
    g = torch.Generator().manual_seed(len(lengths) + d)
    n_pages = sum(-(-n // page) + 1 for n in lengths) + 2
    slots = _runs(lengths, page, g, n_pages)
    qkv = torch.randn((len(slots), Hq + 2 * Hkv, d), generator=g).to(DT[kind])
    _check_append(Cache(n_pages, page, Hkv, d, g), qkv, slots, Hq, Hkv, kind,
                  k_norm=torch.ones(d), rope=kda.rope_table(64, 32, device="cpu"),
                  positions=torch.randint(0, 64, (len(slots),), generator=g).int())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T", [4863, 4865, 9727, 9729, 65700])
def test_append_long_prompts(kind, T):
    """Lengths on either side of those where rows and units of a CTA change."""
    g = torch.Generator().manual_seed(T)
    lengths = [T // 3, 1, 17, T - T // 3 - 18]
    n_pages = sum(-(-n // 128) + 1 for n in lengths)
    slots = _runs(lengths, 128, g, n_pages)
    qkv = torch.randn((T, 4, 64), generator=g).to(DT[kind])
    _check_append(Cache(n_pages, 128, 1, 64, g), qkv, slots, 2, 1, kind, q_norm=torch.ones(64),
                  rope=kda.rope_table(64, 32, device="cpu"),
                  positions=torch.randint(0, 64, (T,), generator=g).int())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_append_magnitudes(kind):
    """Blocks that outgrow their scale by anything, blocks far below it, zeros, values
    at the borders of a scale, values beyond the largest and below the smallest scale."""
    g = torch.Generator().manual_seed(9)
    Hq, Hkv, d, page = 2, 2, 64, 16
    sizes = [2.0 ** -140 if kind == "f32" else 2.0 ** -120, 2.0 ** -60, 2.0 ** -45, 2.0 ** -20, 1.0,
             2.0 ** 20, 2.0 ** 45, 2.0 ** 57]
    slots = _runs([1, 5, 16] * len(sizes), page, g, 100)
    qkv = torch.randn((len(slots), Hq + 2 * Hkv, d), generator=g).double()
    at = 0
    for i, n in enumerate([1, 5, 16] * len(sizes)):
        qkv[at:at + n] *= sizes[i // 3]
        at += n
    qkv[3, 2:] = 0
    qkv[30, 3:, 7] = 448 * 2.0 ** -3          # a scale's border, and the first value above it
    qkv[31, 3:, 7] = 450 * 2.0 ** 1
    qkv = qkv.clamp(-448 * 2.0 ** 50, 448 * 2.0 ** 50).to(DT[kind])
    _check_append(Cache(100, page, Hkv, d, g), qkv, slots, Hq, Hkv, kind)


def test_append_a_nan_is_kept_and_infinities_are_the_largest_value():
    g = torch.Generator().manual_seed(2)
    cache = Cache(3, 16, 1, 64, g)
    qkv = torch.randn((4, 3, 64), generator=g).to(BF16)
    qkv[1, 1:, 5] = float("nan")
    clean = qkv.clone()
    clean[1, 1:, 5] = 0
    slots = torch.tensor([16, 17, 18, 19])
    _, pages, scales, status = _append(cache, qkv, slots, 1, 1)
    _, p0, s0, _ = _append(cache, clean, slots, 1, 1)
    assert status == (kda.KDA_OK, 0)
    for p, q, s, r in zip(pages, p0, scales, s0):
        assert torch.equal(s, r)
        assert p[1, 1, 0, 5].float().isnan()
        a, b = p.view(torch.uint8).clone(), q.view(torch.uint8).clone()
        a[1, 1, 0, 5] = b[1, 1, 0, 5] = 0
        assert torch.equal(a, b)
    qkv = clean.clone()
    qkv[2, 2, 9] = float("inf")
    _, pages, scales, _ = _append(cache, qkv, slots, 1, 1)
    assert float(scales[1][1, 0, 0]) == 2.0 ** 50 and float(pages[1][1, 2, 0, 9].float()) == 448


def test_append_token_by_token_and_at_once():
    """The same tokens one call at a time: a scale of the same size, and values that
    differ by the rounding again of what was there."""
    g = torch.Generator().manual_seed(3)
    Hkv, d, page = 2, 64, 32
    slots = torch.arange(32, 64)
    qkv = torch.randn((32, 3 * Hkv, d), generator=g) * torch.exp2(torch.linspace(-4, 4, 32))[:, None, None]
    qkv = qkv.to(BF16)
    cache = Cache(3, page, Hkv, d, g)
    _, at_once, s1, _ = _append(cache, qkv, slots, Hkv, Hkv)
    for t in range(32):
        _, cache.pages, cache.scales, status = _append(cache, qkv[t:t + 1], slots[t:t + 1], Hkv, Hkv)
        assert status == (kda.KDA_OK, 0)
    for i in range(2):
        assert torch.equal(cache.scales[i][1], s1[i][1])
        a, b = (p[i].double() * spread(s) for p, s in ((cache.pages, s1[i]), (at_once, s1[i])))
        # rounded again with a scale that grew by powers of two: below 2^-6 s each of up to
        # nine roundings is off by half a step 2^-10 s, above it by nothing more
        step = 2.0 ** -10 * spread(s1[i])
        assert ((a - b)[1].abs() <= (9 * step + 2.0 ** -3 * (b.abs() < 2.0 ** -6 * spread(s1[i])) * b.abs())[1]).all()


def test_append_skips_padding_and_bad_tokens():
    """Padding inside a block, slots beyond the pool, positions beyond the table."""
    g = torch.Generator().manual_seed(4)
    Hq, Hkv, d, page = 2, 2, 128, 16
    cache = Cache(6, page, Hkv, d, g)
    T = 40
    slots = torch.cat([torch.arange(20, 40), torch.full((3,), -1), torch.arange(80, 96),
                       torch.tensor([-7])])
    slots[5], slots[25] = -1, -1               # holes in runs
    qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=g).to(BF16)
    _check_append(cache, qkv, slots, Hq, Hkv, "bf16")
    bad = slots.clone()
    bad[7] = 96
    _, pages, scales, status = _append(cache, qkv, bad, Hq, Hkv)
    assert status == (kda.KDA_ERR_DEVICE_CHECK, 1)
    skip = slots.clone()
    skip[7] = -1
    _, p0, s0, _ = _append(cache, qkv, skip, Hq, Hkv)
    rope, pos = kda.rope_table(64, 64, device="cpu"), torch.arange(T).int()
    for x, y in zip(pages + scales, p0 + s0):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    pos_bad = pos.clone()
    pos_bad[7] = 64
    _, pages, scales, status = _append(cache, qkv, slots, Hq, Hkv, rope=rope, positions=pos_bad)
    assert status == (kda.KDA_ERR_DEVICE_CHECK, 1024)
    _, p0, s0, _ = _append(cache, qkv, skip, Hq, Hkv, rope=rope, positions=pos)
    for x, y in zip(pages + scales, p0 + s0):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("order", ["backwards", "shuffled"])
def test_append_tokens_of_a_block_in_any_order(order):
    """Rows of a block within 16 of one another need not be in order."""
    g = torch.Generator().manual_seed(12)
    cache = Cache(5, 16, 2, 64, g)
    runs = [torch.arange(16, 32), torch.arange(37, 45), torch.arange(70, 71)]
    if order == "backwards":
        runs = [r.flip(0) for r in runs]
    else:
        runs = [r[torch.randperm(len(r), generator=g)] for r in runs]
    slots = torch.cat(runs)
    qkv = torch.randn((len(slots), 6, 64), generator=g).to(BF16)
    _check_append(cache, qkv, slots, 2, 2, "bf16")


@pytest.mark.parametrize("bad", [float("nan"), 0.0, -2.0, float("inf"), 2.0 ** 51])
def test_append_old_scales_outside_their_range(bad):
    """A continued block's scale that is none counts as the smallest one; a block that
    starts anew does not look at it."""
    g = torch.Generator().manual_seed(5)
    cache = Cache(4, 16, 1, 64, g)
    slots = torch.tensor([19, 20, 32])
    qkv = torch.randn((3, 3, 64), generator=g).to(BF16)
    for s in cache.scales:
        s[1:3] = bad
    _, _, scales, status = _append(cache, qkv, slots, 1, 1)
    assert status == (kda.KDA_ERR_DEVICE_CHECK, 8192)
    for i, x in enumerate((qkv[:, 1], qkv[:, 2])):
        assert float(scales[i][1, 0, 0]) == float(scale_for(x[:2].abs().max()))
        assert float(scales[i][2, 0, 0]) == float(scale_for(x[2].abs().max()))


def _borders(d, ties):
    """d numbers between two neighbouring e4m3 values each (ties), from 2^-10 to 2^7."""
    at = torch.arange(d)
    e = (at // 8 % 16 - 8).double()
    x = (8 + at % 8 + (0.5 if ties else 0.0)) / 8 * torch.exp2(e)
    low = (at % 8 + 8 * (e + 8) + 0.5) * 2.0 ** -9      # below 2^-6 the grid is even
    return torch.where(e < -6, low, x)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_append_into_scales_that_are_no_powers_of_two(kind, d):
    """A continued block may have any scale: new values that lie on a border between two
    e4m3 values when divided by it, or (fp32) next to one, are stored as the exact
    quotient's rounding."""
    g = torch.Generator().manual_seed(d)
    Hkv, page, n = 2, 16, 128                  # a block each
    cache = Cache(n, page, Hkv, d, g)
    m = torch.arange(128, 256).double() / 128 if kind == "bf16" else 1 + torch.rand(128, generator=g).double()
    tokens = 3
    slots = (torch.arange(n)[:, None] * page + torch.tensor([3, 4, 5])).flatten()
    qkv = torch.zeros((n * tokens, 3 * Hkv, d), dtype=DT[kind])
    for i in range(2):
        scale = torch.stack([m[torch.randperm(128, generator=g)] * 2.0 ** (3 * h - 4 + i) for h in range(Hkv)], 1)
        cache.scales[i][:, 0] = scale.float()
        x = (cache.scales[i][:, 0].double()[..., None] * _borders(d, True)).to(DT[kind])
        off = x, torch.nextafter(x.float(), torch.tensor(1e9)), torch.nextafter(x.float(), torch.tensor(0.0))
        for k in range(tokens):
            qkv[k::tokens, (1 + i) * Hkv:(2 + i) * Hkv] = off[k].to(DT[kind])
    _check_append(cache, qkv, slots, Hkv, Hkv, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_append_grows_scales_that_are_no_powers_of_two(kind):
    """Old scales whose products with an e4m3 value lie next to a border between two
    others, nearer than an fp32 product tells: rounded again as the exact product."""
    g = torch.Generator().manual_seed(8)
    Hkv, d, page = 2, 64, 16
    odd = torch.arange(17, 32, 2).double()
    scales = torch.cat([torch.round(odd * 2.0 ** 23 / y) + o for y in (9.0, 11.0, 13.0, 15.0) for o in (-1, 0, 1)])
    scales = scales[(scales >= 2.0 ** 23) & (scales < 2.0 ** 24)] * 2.0 ** -23
    n = len(scales)
    cache = Cache(n, page, Hkv, d, g)
    for i in range(2):
        byte = torch.randint(0, 127, (n, page, Hkv, d), generator=g) + 128 * torch.randint(0, 2, (n, page, Hkv, d), generator=g)
        cache.pages[i] = byte.to(torch.uint8).view(E4M3)
        for h in range(Hkv):
            cache.scales[i][:, 0, h] = scales[torch.randperm(n, generator=g)].float()
    slots = torch.arange(n) * page + 15
    qkv = torch.randn((n, 3 * Hkv, d), generator=g)
    qkv[..., 7] = (448 * torch.exp2(1 + torch.arange(n) % 3))[:, None]     # grows to 2, 4 or 8
    _check_append(cache, qkv.to(DT[kind]), slots, Hkv, Hkv, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_append_beyond_32_bit_offsets(kind):
    """A pool and a batch of more than 2^31 elements."""
    Hq, Hkv, d, page = 14, 1, 128, 256
    T = (1 << 31) // ((Hq + 2 * Hkv) * d) + 100
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.zeros((T, Hq + 2 * Hkv, d), dtype=DT[kind], device="cuda")
    qkv[-50:] = torch.randn((50, Hq + 2 * Hkv, d), generator=g, device="cuda").to(DT[kind])
    n_pages = (1 << 32) // (page * Hkv * d) + 3
    slot = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    slot[-50:] = torch.arange(50, device="cuda", dtype=torch.int32) + (n_pages - 1) * page + 3
    pages = [torch.zeros((n_pages, page, Hkv, d), dtype=E4M3, device="cuda") for _ in range(2)]
    scales = [torch.full((n_pages, page // BLOCK, Hkv), 2.0 ** -20, device="cuda") for _ in range(2)]
    q = torch.zeros((T, Hq, d), dtype=DT[kind], device="cuda")
    ws = kda.paged_workspace_for()
    kda.kda_paged_append_q8(qkv, None, None, None, None, slot, q, *pages, *scales, workspace=ws)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    assert torch.equal(q[-50:], qkv[-50:, :Hq]) and not q[:-50].any()
    x = qkv[-50:, Hq:].cpu().double()
    for i in range(2):
        got = pages[i][-1].cpu().double() * spread(scales[i][-1].cpu())
        for b in range(4):
            rows = slice(max(0, 16 * b - 3), min(50, 16 * b + 13))
            s = float(scale_for(x[rows, i].abs().max()))
            assert float(scales[i][-1, b, 0]) == s
            assert torch.equal(got[3:53][rows, 0], rounded(x[rows, i] / s) * s)
        assert not pages[i][:-1].view(torch.uint8).any()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mode", ["half", "interleaved"])
def test_queries_of_both_appends(kind, d, mode):
    """q_out of the 8-bit append and of the other: the same formula, each with fp32's
    errors (as in _check_append) and one rounding."""
    g = torch.Generator().manual_seed(d)
    Hq, Hkv, T, rot = 6, 2, 90, 48
    qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=g).to(DT[kind])
    slots, pos = torch.arange(16, 16 + T), torch.randint(0, 500, (T,), generator=g).int()
    norms = [1 + 0.1 * torch.randn(d, generator=g) for _ in range(2)]
    rope = kda.rope_table(500, rot, device="cpu")
    q, *_ = _append(Cache(8, 16, Hkv, d, g), qkv, slots, Hq, Hkv, q_norm=norms[0], k_norm=norms[1],
                    rope=rope, positions=pos, mode=mode)
    pages = [torch.zeros((8, 16, Hkv, d), dtype=DT[kind], device="cuda") for _ in range(2)]
    other = torch.empty((T, Hq, d), dtype=DT[kind], device="cuda")
    ws = kda.paged_workspace_for()
    kda.kda_paged_append(qkv.cuda(), norms[0].cuda(), norms[1].cuda(), rope.cuda(), pos.cuda(),
                         slots.int().cuda(), other, *pages, rope_mode=mode, workspace=ws)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    (ref, size), _, _ = append_reference(qkv, *norms, rope, pos, Hq, Hkv, mode, 1e-6)
    u, half = half_step(F32), half_step(DT[kind])
    off = 2 * (half * ref.abs() * 1.01 + (d + 16) * u * size * 2) + 1e-30
    assert ((q.double() - other.double().cpu()).abs() <= off).all()


def test_append_zero_tokens():
    g = torch.Generator().manual_seed(5)
    cache = Cache(2, 16, 1, 64, g)
    _append(cache, torch.zeros((0, 3, 64), dtype=BF16), torch.zeros(0), 1, 1)
    assert kda.kda_last_launch_count() == 0


def test_append_in_a_graph_on_another_stream_leaves_the_same():
    """A captured append replayed: the scales have grown, and the second pass changes
    nothing more."""
    g = torch.Generator().manual_seed(15)
    cache = Cache(8, 32, 2, 128, g)
    slots = _runs([1, 20, 1, 33], 32, g, 8)
    qkv = torch.randn((len(slots), 8, 128), generator=g).to(BF16)
    q0, p0, s0, _ = _append(cache, qkv, slots, 4, 2)
    t = [x.cuda() for x in (qkv, slots.int())]
    pages, scales = [x.cuda() for x in cache.pages], [x.cuda() for x in cache.scales]
    q, ws = torch.zeros_like(q0).cuda(), kda.paged_workspace_for()
    call = lambda: kda.kda_paged_append_q8(t[0], None, None, None, None, t[1], q, *pages, *scales,
                                           workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q.cpu(), q0)
        for x, y in zip(pages + scales, p0 + s0):
            assert torch.equal(x.cpu().view(torch.uint8), y.view(torch.uint8))
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)


# -------------------------------------------------------------------- together

def test_serving_steps_together():
    """Prompts, then decode steps, over one 8-bit cache: plan, append, attention, the
    step's log probabilities and the verification of a draft.  The attention is that of
    the values that went in, off by their rounding to e4m3."""
    g = torch.Generator().manual_seed(77)
    Hq, Hkv, d, page, n_pages, B, V = 4, 2, 64, 16, 40, 3, 997
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pages = [torch.full((n_pages, page, Hkv, d), NAN8, dtype=torch.uint8, device="cuda").view(E4M3)
             for _ in range(2)]
    scales = [torch.full((n_pages, 1, Hkv), float("nan"), device="cuda") for _ in range(2)]
    table, ring, state = i32([[0] * 12] * B), i32(list(range(n_pages))), i32([0, n_pages])
    held, cached = i32([0] * B), [0] * B
    keys, values = [torch.zeros(0, Hkv, d)] * B, [torch.zeros(0, Hkv, d)] * B
    rope = kda.rope_table(256, d)
    head = torch.randn((Hq * d, V), generator=g)
    for new in ([50, 1, 17], [1, 1, 1], [1, 4, 0], [1, 1, 1]):
        T = sum(new)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=g).to(BF16)
        held_out, state_out, kv = i32([0] * B), i32([0, 0]), i32([0] * B)
        pos, slot, q = i32([0] * T), i32([0] * T), torch.zeros((T, Hq, d), dtype=BF16, device="cuda")
        ws = kda.paged_workspace_for(T, Hq, Hkv, d)
        kda.kda_paged_plan(i32(cu), i32(cached), table, held, ring, state, held_out, state_out, kv,
                           pos, slot, page_size=page, workspace=ws)
        kda.kda_paged_append_q8(qkv.cuda(), None, None, rope, pos, slot, q, *pages, *scales,
                                workspace=ws)
        out = torch.zeros_like(q)
        kda.kda_paged_attn_q8(q, *pages, *scales, table, i32(cu), kv, out, workspace=ws)
        assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
        _, (rk, _), rv = append_reference(qkv, None, None, rope.cpu(), pos.cpu(), Hq, Hkv, "half", 0)
        got, qc = out.double().cpu(), q.double().cpu()
        for b, n in enumerate(new):
            keys[b] = torch.cat([keys[b], rk[cu[b]:cu[b + 1]]])
            values[b] = torch.cat([values[b], rv[cu[b]:cu[b + 1]]])
            for i in range(n):
                t, seen = cu[b] + i, cached[b] + i + 1
                for h in range(Hq):
                    K, W = keys[b][:seen, h // 2].double(), values[b][:seen, h // 2].double()
                    s = K @ qc[t, h] / d ** 0.5
                    # a key's channels are off by 2^-4 of themselves and by what a scale that
                    # grew rounded again (the largest times 2^-15): the score by e, the
                    # weights by expm1(2 e), the values by 2^-4 and their tiny share
                    e = float((2.0 ** -4 * (K.abs() @ qc[t, h].abs())
                               + 2.0 ** -12 * qc[t, h].abs().sum()).max()) / d ** 0.5
                    w = torch.softmax(s, 0)
                    size = w @ W.abs()
                    off = size * (torch.expm1(torch.tensor(2 * e)) * 1.07 + 2.0 ** -4 + 2.0 ** -7) + 2.0 ** -10
                    assert ((got[t, h] - w @ W).abs() <= off).all()
        last = [c - 1 for c, n in zip(cu[1:], new) if n]
        logits = (got[last].flatten(1).float() @ head).cuda()
        N = len(last)
        f = lambda *s: torch.zeros(s, device="cuda")
        lp, ent, rank, ids, top = f(N), f(N), i32([0] * N), i32([[0] * 3] * N), f(N, 3)
        tok = logits.argmax(-1).int()
        kda.kda_token_logprobs(logits, tok, lp, ent, rank, ids, top, workspace=ws)
        assert rank.tolist() == [0] * N and torch.equal(ids[:, 0], tok) and torch.equal(top[:, 0], lp)
        probs = torch.softmax(logits, -1)[:, None].contiguous()
        accepted, tokens = i32([0] * N), i32([[0]] * N)
        kda.kda_verify_drafts(probs, None, i32([[]] * N), f(N, 0), f(N), accepted, tokens, workspace=ws)
        assert accepted.tolist() == [1] * N
        assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
        cached, held, state = [c + n for c, n in zip(cached, new)], held_out, state_out
