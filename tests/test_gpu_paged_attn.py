"""GPU parity of kda_paged_attn with a 64-bit plain form: one token to long
chunks, odd lengths and tile borders, every page size and group size, rows that
see nothing, pages that end inside a tile, poisoned memory around the keys;
determinism, graphs and the device-side checks."""

import pytest
import torch

import hybrid_linear_attention_delta_gb300 as kda
from kda_cases import TOL
from paged_cases import AttnCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.lib()


def _run(case, causal=True, scale=None, dev=None, ws=None, out=None):
    t = dev or case.cuda()
    if out is None:
        out = torch.full_like(t["q"], AttnCase.MARK)
    if ws is None:
        ws = kda.paged_workspace_for(t["q"].shape[0], case.Hq, case.Hkv, case.d)
    kda.kda_paged_attn(t["q"], t["k"], t["v"], t["table"], t["cu"], t["kv"], out, scale=scale,
                       causal=causal, workspace=ws)
    return out, ws


def _check(case, causal=True, scale=None, norm_bar=True):
    out, ws = _run(case, causal, scale)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    assert kda.kda_last_launch_count() == 1
    used = int(case.cu[-1])
    ref, size, top = case.reference(causal, scale)
    got = out.double().cpu()
    assert torch.isfinite(got).all()
    err = (got - ref)[:used].abs()
    over = err > case.bound(ref, size, top)[:used]
    assert not over.any(), (float(err.max()), int(over.sum()), over.nonzero()[:4].tolist())
    name = "bf16" if case.dtype == torch.bfloat16 else "f32"
    if norm_bar and used and float(ref.norm()) > 0:
        assert float((got - ref)[:used].norm() / ref.norm()) <= TOL[name]
    assert (out[used:] == AttnCase.MARK).all()          # rows behind the last request
    assert int(ws[256:256 + 8 * 152].sum()) == 0        # counters are left as they were found
    return out


LENGTHS = [
    ([1], [1]), ([1], [777]), ([1, 1, 1], [127, 128, 129]), ([5], [5]), ([64], [200]),
    ([130], [130]), ([1, 0, 7, 33], [40, 0, 7, 300]), ([200, 3], [200, 1000]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,total", LENGTHS)
def test_lengths(dtype, d, new, total):
    _check(AttnCase(new, total, Hq=8, Hkv=2, d=d, page=16, dtype=dtype, seed=len(new), pad=3))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(dtype, page):
    _check(AttnCase([70, 1, 9], [333, 257, 256], Hq=4, Hkv=2, d=128, page=page, dtype=dtype,
                    seed=page))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (3, 1), (10, 2), (7, 1), (16, 1), (24, 1),
                                    (64, 1), (33, 3)])
def test_groups(dtype, Hq, Hkv):
    """Groups that fill a tile of rows and groups that leave some of it empty."""
    _check(AttnCase([43, 1, 150], [300, 200, 151], Hq=Hq, Hkv=Hkv, d=64, page=32, dtype=dtype,
                    seed=Hq))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing(dtype, causal):
    """No keys at all, and more new tokens than keys: their rows are zeros."""
    case = AttnCase([4, 9, 1, 300], [0, 3, 50, 20], Hq=6, Hkv=2, d=64, page=16, dtype=dtype)
    out = _check(case, causal)
    assert (out[:4] == 0).all()
    if causal:
        assert (out[4:10] == 0).all() and (out[10:13] != 0).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_not_causal_and_scale(dtype):
    case = AttnCase([40, 1], [500, 77], Hq=4, Hkv=1, d=128, page=64, dtype=dtype)
    _check(case, causal=False)
    _check(case, scale=0.02)
    _check(case, scale=0.0)
    _check(case, scale=-0.05)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_smallest_scales(dtype):
    """Queries and keys so large that their products need a scale of 10^-34, and a
    scale of zero whatever the products."""
    case = AttnCase([40, 1], [500, 77], Hq=4, Hkv=1, d=64, page=64, dtype=dtype, seed=2)
    case.q, case.k = (x.double().mul(2.0 ** 56).to(case.dtype) for x in (case.q, case.k))
    _check(case, scale=2.0 ** -115)
    _check(case, scale=-2.0 ** -115)
    _check(case, scale=0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 128), (8, 1, 128), (16, 8, 64)])
def test_long_context_is_split_and_joined(dtype, Hq, Hkv, d):
    """Few rows over many keys: pieces on every SM, joined in order."""
    case = AttnCase([1], [20011], Hq=Hq, Hkv=Hkv, d=d, page=16, dtype=dtype, seed=5)
    a = _check(case)
    b, _ = _run(case)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,new", [(3, 1), (4, 1), (5, 1), (8, 2), (17, 1), (64, 2), (7, 30)])
def test_pieces_are_joined_whatever_the_rows(dtype, d, G, new):
    """One item over some twenty CTAs: no more rows than a warp each, a few, a
    tile of them, two tiles; and two heads, so that pieces of both are about."""
    _check(AttnCase([new, 1], [9001, 130], Hq=2 * G, Hkv=2, d=d, page=64, dtype=dtype, seed=G))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores(dtype):
    """Scores that differ by hundreds: the running maximum moves often and a few
    keys carry all the weight.  (A score of 300 is summed to 300 half steps of
    fp32, which the element bound counts and the norm's bar does not.)"""
    case = AttnCase([50, 1], [700, 2900], Hq=4, Hkv=2, d=64, page=16, dtype=dtype, seed=9,
                    scale_q=40.0)
    _check(case, norm_bar=False)


def test_rising_scores_move_the_maximum_every_tile():
    """Keys whose score grows along the sequence, so that every tile has a new
    maximum far above the last one, and keys that fall, so that none has."""
    for sign in (1.0, -1.0):
        case = AttnCase([130], [1500], Hq=2, Hkv=1, d=64, page=16, dtype="bf16", seed=3)
        ramp = sign * torch.linspace(-40, 40, 1500)
        ids = case.table[0].long()
        k = case.k[ids].reshape(-1, 1, 64)
        k[:1500, :, 0] = ramp[:, None].to(torch.bfloat16)
        case.k[ids] = k.reshape(-1, 16, 1, 64)
        case.q[..., 0] = 6.0
        _check(case, norm_bar=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,new,total", [
    (2, 1, [130], [1500]),            # two tiles of rows
    (4, 2, [300, 1, 0, 9], [900, 2900, 5, 640]),  # both forms of item, ragged ends
    (8, 1, [1], [20011]),             # one item over many CTAs
    (64, 1, [5], [6000]),             # both tiles of rows over many CTAs
])
@pytest.mark.parametrize("kind", ["rising", "falling", "steps", "large"])
def test_references_move(d, Hq, Hkv, new, total, kind):
    """Scores that pass a row's reference: from tile to tile, in jumps that are
    apart from one row to the next, or anywhere (sums and outputs are rescaled, the
    tile's weights made again), and scores that fall, where nothing moves."""
    case = AttnCase(new, total, Hq=Hq, Hkv=Hkv, d=d, page=16, dtype="bf16", seed=d + Hq,
                    scale_q=30.0 if kind == "large" else 1.0)
    for b, t in enumerate(total if kind != "large" else []):
        if t == 0:
            continue
        at = torch.arange(t, dtype=torch.float64)
        ramp = {"rising": -40 + 80 * at / t, "falling": 40 - 80 * at / t,
                "steps": 10.0 * (at // 200)}[kind]
        ids = case.table[b, :-(-t // 16)].long()
        k = case.k[ids].reshape(-1, Hkv, d)
        k[:t, :, 0] = ramp[:, None].to(torch.bfloat16)
        case.k[ids] = k.reshape(-1, 16, Hkv, d)
    if kind != "large":
        rows = torch.arange(case.q.shape[0])[:, None] % 3
        case.q[..., 0] = (torch.tensor([6.0, 0.5, 20.0])[rows]).to(torch.bfloat16)
    _check(case, norm_bar=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,total,hidden", [
    ([3, 1], [700, 300], 300), ([1], [9000], 4097),   # few rows, cut items
    ([1] * 40, [1000] * 40, 500),                     # few rows, key tiles in turn
    ([300, 70], [1500, 900], 600),                    # two tiles of rows
])
def test_scores_of_minus_infinity_before_others(dtype, d, new, total, hidden):
    """Keys that a row scores -inf fill its first tiles; the others' scores are far
    below zero and carry all the weight."""
    Hkv = 8 if len(new) > 2 else 2
    case = AttnCase(new, total, Hq=8, Hkv=Hkv, d=d, page=16, dtype=dtype, seed=hidden + d)
    for b, t in enumerate(total):
        ids = case.table[b, :-(-t // 16)].long()
        k = case.k[ids].reshape(-1, Hkv, d)
        k[:t, :, 0] = 0.0
        k[:t, :, 1] = -40.0
        k[:min(hidden, t - 1), :, 0] = -float("inf")
        case.k[ids] = k.reshape(-1, 16, Hkv, d)
    case.q[..., 0], case.q[..., 1] = 1.0, 6.0 * d ** 0.5
    ref, size, _ = case.reference()
    out, ws = _run(case)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    case.k = torch.where(case.k == -float("inf"), torch.zeros_like(case.k), case.k)
    _, _, top = case.reference()            # sum |q k| of the keys with finite scores
    got = out.double().cpu()
    assert ((got - ref).abs() <= case.bound(ref, size, top)).all(), float((got - ref).abs().max())


def test_mixed_batch_of_many_requests():
    g = torch.Generator().manual_seed(11)
    new = torch.randint(0, 60, (90,), generator=g).tolist()
    total = [n + c for n, c in zip(new, torch.randint(0, 400, (90,), generator=g).tolist())]
    _check(AttnCase(new, total, Hq=6, Hkv=2, d=128, page=16, dtype="bf16", seed=12, pad=17))


def test_chunk_against_a_long_prefix():
    _check(AttnCase([519], [4100], Hq=8, Hkv=2, d=128, page=128, dtype="bf16", seed=21))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_beyond_32_bit_offsets(dtype):
    """A pool of more than 2^31 elements, with the request's pages at its end."""
    Hkv, d, page = 8, 128, 256
    case = AttnCase([3, 1], [600, 90], Hq=8, Hkv=Hkv, d=d, page=page, dtype=dtype, seed=4)
    t = case.cuda()
    n_small = case.k.shape[0]
    n_pages = (1 << 31) // (page * Hkv * d) + 40
    big = {}
    for n in ("k", "v"):
        big[n] = torch.zeros((n_pages, page, Hkv, d), dtype=case.dtype, device="cuda")
        big[n][n_pages - n_small:] = t[n]
    t.update(big)
    t["table"] = t["table"] + (n_pages - n_small)
    out, _ = _run(case, dev=t)
    ref, size, top = case.reference()
    assert ((out.double().cpu() - ref).abs() <= case.bound(ref, size, top)).all()


@pytest.mark.parametrize("d,Hkv,G,B,T,lg", [
    (128, 16, 2, 1, 1280, 22),   # items of whole tiles of rows, each on one CTA
    (64, 16, 3, 1, 1000, 22),
    (128, 4, 4, 40, 1, 24),      # decodes: an item and a part of one on a CTA
    (64, 4, 4, 40, 1, 24),
    (128, 2, 8, 1, 2, 26),       # an item over many CTAs, several runs on each
])
@pytest.mark.parametrize("causal", [True, False])
def test_sums_over_millions_of_keys(d, Hkv, G, B, T, lg, causal):
    """Values of one sign, whose sums in tensor memory would lose 1e-2 and more to
    the products that are cut off.  The pages of a request are the same sixteen
    over and over: every distinct key weighs as often, but for the few at the end that
    a row of the causal forms does not see (1282 of 2^22 at most)."""
    g = torch.Generator(device="cuda").manual_seed(lg + d)
    page, n_pages, kv = 256, 16, (1 << lg) - (3 if causal else 0)
    k = torch.randn((n_pages, page, Hkv, d), generator=g, device="cuda").bfloat16()
    v = (torch.randn((n_pages, page, Hkv, d), generator=g, device="cuda").abs() + 0.5).bfloat16()
    q = torch.randn((B * T, Hkv * G, d), generator=g, device="cuda").bfloat16()
    table = (torch.arange(1 << lg - 8, device="cuda") % n_pages).int().repeat(B, 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ws = kda.paged_workspace_for(B * T, Hkv * G, Hkv, d)
    outs = []
    for _ in range(2):
        out = torch.zeros_like(q)
        kda.kda_paged_attn(q, k, v, table, i32([T * b for b in range(B + 1)]), i32([kv] * B), out,
                           causal=causal, workspace=ws)
        assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
        outs.append(out)
    assert torch.equal(*outs)
    ref = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for h in range(Hkv * G):
        K, V = (x[:, :, h // G].flatten(0, 1).double() for x in (k, v))
        ref[:, h] = torch.softmax(q[:, h].double() @ K.T * d ** -0.5, -1) @ V
    # weights and outputs are rounded to bf16; a run of 2^17 keys loses at most 2^-26
    # of its sum per key, on average over the run half of that: 2^-10.  (The keys that
    # a causal row does not see are 3e-4 of all, but may weigh many times the mean: those
    # forms are compared by their norm alone.)
    err = outs[0].double() - ref
    if not causal:
        assert (err.abs() <= ref.abs() * (2 * 2.0 ** -8 * 1.01 + 2.0 ** -10)).all()
    assert float(err.norm() / ref.norm()) <= TOL["bf16"]


def test_exact_sums_over_2_to_27_keys():
    """Keys of zeros weigh the same and values are powers of two, so that every sum
    is exact as long as it is kept: the outputs are the values."""
    Hq, d, page, kv, T = 64, 64, 256, 1 << 27, 640
    q = torch.ones((T, Hq, d), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((1, page, 1, d), dtype=torch.bfloat16, device="cuda")
    value = 2.0 ** (torch.arange(d, device="cuda") % 5)
    v = value.to(torch.bfloat16).expand(1, page, 1, d).contiguous()
    table = torch.zeros((1, kv // page), dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ws = kda.paged_workspace_for(T, Hq, 1, d)
    out = torch.zeros_like(q)
    kda.kda_paged_attn(q, k, v, table, i32([0, T]), i32([kv]), out, causal=False, workspace=ws)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    assert (out.float() == value).all()


def test_captured_graphs_share_a_workspace_and_follow_the_lengths():
    """Two graphs over one workspace, replayed in turn with other lengths."""
    cases = [AttnCase([1, 1], [900, 300], Hq=8, Hkv=2, d=128, page=16, dtype="bf16", seed=1),
             AttnCase([40, 9], [140, 2000], Hq=8, Hkv=2, d=128, page=32, dtype="bf16", seed=2)]
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
        ref, size, top = c.reference()
        assert ((o.double().cpu() - ref).abs() <= c.bound(ref, size, top)).all()
    # shorter requests in the captured call
    cases[0].total = [500, 17]
    devs[0]["kv"].copy_(torch.tensor([500, 17], dtype=torch.int32))
    graphs[0].replay()
    ref, size, top = cases[0].reference()
    assert ((outs[0].double().cpu() - ref).abs() <= cases[0].bound(ref, size, top)).all()
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)


def test_another_stream():
    case = AttnCase([9], [300], Hq=4, Hkv=2, d=64, page=16, dtype="bf16")
    t = case.cuda()
    s = torch.cuda.Stream()
    ws = kda.paged_workspace_for(9, 4, 2, 64)
    out = torch.zeros_like(t["q"])
    s.wait_stream(torch.cuda.current_stream())
    kda.kda_paged_attn(t["q"], t["k"], t["v"], t["table"], t["cu"], t["kv"], out, workspace=ws,
                       stream=s)
    s.synchronize()
    ref, size, top = case.reference()
    assert ((out.double().cpu() - ref).abs() <= case.bound(ref, size, top)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_short_requests(dtype):
    """More requests than threads of a CTA, most of them a token, some of them
    without one."""
    g = torch.Generator().manual_seed(31)
    new = torch.randint(0, 3, (1500,), generator=g).tolist()
    total = [n + c for n, c in zip(new, torch.randint(0, 40, (1500,), generator=g).tolist())]
    _check(AttnCase(new, total, Hq=2, Hkv=1, d=64, page=16, dtype=dtype, seed=32, pad=5))


@pytest.mark.parametrize("d", [64, 128])
def test_f32_counters_of_every_cta_are_left_at_zero(d):
    """Cut items all over the line: the counters of all CTAs, 304 of them with 64
    channels, are as they were found, and the next call joins as this one did."""
    case = AttnCase([1, 3, 1, 40] * 5, [9000, 4000, 2500, 3100] * 5, Hq=16, Hkv=8, d=d, page=32,
                    dtype="f32", seed=d)
    t = case.cuda()
    first, ws = _run(case, dev=t)
    assert int(ws[256:256 + 8 * 304].sum()) == 0
    ref, size, top = case.reference()
    assert ((first.double().cpu() - ref).abs() <= case.bound(ref, size, top)).all()
    for _ in range(3):
        again, _ = _run(case, dev=t, ws=ws)
        assert torch.equal(again, first)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own, in flight together."""
    cases = [AttnCase([1, 40], [3000, 700], Hq=8, Hkv=2, d=d, page=16, dtype="bf16", seed=d)
             for d in (64, 128)]
    devs = [c.cuda() for c in cases]
    outs = [torch.zeros_like(t["q"]) for t in devs]
    wss = [kda.paged_workspace_for(41, 8, 2, c.d) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, t, o, ws, s in zip(cases, devs, outs, wss, streams):
            kda.kda_paged_attn(t["q"], t["k"], t["v"], t["table"], t["cu"], t["kv"], o,
                               workspace=ws, stream=s)
    torch.cuda.synchronize()
    for c, o, ws in zip(cases, outs, wss):
        ref, size, top = c.reference()
        assert ((o.double().cpu() - ref).abs() <= c.bound(ref, size, top)).all()
        assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,d", [(8, 128), (3, 64)])
def test_out_over_q(dtype, G, d):
    """The outputs take the queries' place: whole items, two tiles of rows, and
    items whose pieces lie on many CTAs."""
    case = AttnCase([1, 90, 0, 301, 2], [9000, 700, 5, 301, 4000], Hq=2 * G, Hkv=2, d=d, page=32,
                    dtype=dtype, seed=G)
    apart, _ = _run(case)
    t = case.cuda()
    ws = kda.paged_workspace_for(t["q"].shape[0], 2 * G, 2, d)
    kda.kda_paged_attn(t["q"], t["k"], t["v"], t["table"], t["cu"], t["kv"], t["q"], workspace=ws)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    assert torch.equal(t["q"], apart)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_pages(dtype):
    """Requests whose rows name the same pages (a shared prompt), and one row
    that names a page twice."""
    case = AttnCase([5, 7], [64, 64], Hq=4, Hkv=2, d=64, page=16, dtype=dtype, seed=6)
    case.table[1, :3] = case.table[0, :3]
    case.table[0, 2] = case.table[0, 0]
    _check(case)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_nan_stays_in_its_row(dtype):
    """A query that holds a NaN gives NaNs, and nothing else does."""
    case = AttnCase([70], [300], Hq=2, Hkv=1, d=64, page=16, dtype=dtype, seed=8)
    clean, _ = _run(case)
    case.q[33, 1, 5] = float("nan")
    out, _ = _run(case)
    assert out[33, 1].isnan().all()
    keep = torch.ones(70, 2, dtype=torch.bool)
    keep[33, 1] = False
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_lengths_tables_and_pages(dtype):
    """Inputs that the device checks refuse: an error bit, and nothing else."""
    mk = lambda: AttnCase([3, 5], [40, 60], Hq=4, Hkv=2, d=64, page=16, dtype=dtype)
    for cu in ([0, 9, 8], [1, 3, 8], [0, 3, 9]):
        case = mk()
        case.cu = torch.tensor(cu, dtype=torch.int32)
        out, ws = _run(case)
        assert kda.kda_device_status(ws) == (kda.KDA_ERR_DEVICE_CHECK, 4)
        assert (out == AttnCase.MARK).all()
    for bad in (-1, 65):     # negative; beyond the table's four pages
        case = mk()
        ref, size, top = case.reference()
        case.kv[1] = bad
        out, ws = _run(case)
        assert kda.kda_device_status(ws) == (kda.KDA_ERR_DEVICE_CHECK, 128)
        assert (out[3:] == AttnCase.MARK).all()
        assert ((out.double().cpu() - ref)[:3].abs() <= case.bound(ref, size, top)[:3]).all()
    for page in (-5, 1 << 20):   # reads as zeros: keys and values 16..31 of request 0
        case = mk()
        good = int(case.table[0, 1])
        t = case.cuda()
        t["table"][0, 1] = page
        case.k[good], case.v[good] = 0, 0
        out, ws = _run(case, dev=t)
        assert kda.kda_device_status(ws) == (kda.KDA_ERR_DEVICE_CHECK, 512)
        ref, size, top = case.reference()
        assert ((out.double().cpu() - ref).abs() <= case.bound(ref, size, top)).all()
