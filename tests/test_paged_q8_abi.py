"""CPU-side checks of the 8-bit cache's calls and of kda_token_logprobs: host-visible
argument errors return before any launch, and the binding's refusals."""

import ctypes

import pytest
import torch

import hybrid_linear_attention_delta_gb300 as kda
from q8_cases import rounded, scale_for

V = ctypes.c_void_p
WS = V(1 << 20)
BAD, UNSUP = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    kda.build()
    return kda.lib()


def _at(n):
    return [V((1 << 24) + (k << 20)) for k in range(n)]


def _args(**kw):
    base = dict(B=2, T_total=8, Hq=4, Hkv=2, d=64, page_size=16, n_pages=8, max_pages=4,
                dtype=kda.KDA_BF16, workspace=WS, workspace_bytes=1 << 23)
    base.update(kw)
    return kda.KdaPagedArgs(**base)


def _attn(lib, ptrs=None, scale=0.1, causal=1, **kw):
    return lib.kda_paged_attn_q8(*(ptrs or _at(9)), scale, causal, ctypes.byref(_args(**kw)))


def _append(lib, ptrs=None, f=None, **kw):
    base = dict(q_norm=V(1 << 28), k_norm=V(1 << 28), rope=V(1 << 29), max_pos=10, rot_dim=32,
                rope_mode=0, norm_eps=1e-6)
    base.update(f or {})
    return lib.kda_paged_append_q8(*(ptrs or _at(8)), ctypes.byref(kda.KdaAppendArgs(**base)),
                                   ctypes.byref(_args(**kw)))


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=7), BAD), (dict(Hq=5), BAD), (dict(Hkv=0), BAD), (dict(d=96), UNSUP),
    (dict(Hq=130), UNSUP), (dict(page_size=8), UNSUP), (dict(n_pages=0), BAD),
    (dict(n_pages=1 << 27), UNSUP), (dict(T_total=-1), BAD), (dict(workspace=None), BAD),
    (dict(workspace=V(1 << 20 | 16)), BAD), (dict(workspace_bytes=128), BAD)])
def test_both_refuse_sizes(lib, kw, want):
    assert _attn(lib, **kw) == want
    assert _append(lib, **kw) == want
    assert lib.kda_last_launch_count() == 0


def test_attention_refuses_pointers_and_scalars(lib):
    for i in range(9):
        for p in (None, V((1 << 24) + 2)):
            ptrs = _at(9)
            ptrs[i] = p
            assert _attn(lib, ptrs) == BAD, i
    for scale in (float("nan"), float("inf"), 2.4e38):
        assert _attn(lib, scale=scale) == BAD
    assert _attn(lib, causal=2) == BAD
    for kw in (dict(max_pages=0), dict(B=-1)):
        assert _attn(lib, **kw) == BAD
    assert _attn(lib, B=8193) == UNSUP
    assert lib.kda_paged_attn_q8(*_at(9), 0.1, 1, None) == BAD
    assert _attn(lib, [None] * 9, B=0) == kda.KDA_OK
    assert _attn(lib, [None] * 9, T_total=0) == kda.KDA_OK
    assert lib.kda_last_launch_count() == 0


def test_append_refuses_pointers_and_scalars(lib):
    for i in range(8):
        for p in (None, V((1 << 24) + 2)):
            ptrs = _at(8)
            ptrs[i] = p
            assert _append(lib, ptrs) == BAD, i
    for f, want in ((dict(rot_dim=-16), BAD), (dict(rot_dim=80), BAD), (dict(rot_dim=24), UNSUP),
                    (dict(rope=None), BAD), (dict(max_pos=0), BAD), (dict(rope_mode=2), BAD),
                    (dict(norm_eps=-1.0), BAD), (dict(q_norm=V(4100)), BAD)):
        assert _append(lib, f=f) == want
    assert lib.kda_paged_append_q8(*_at(8), None, ctypes.byref(_args())) == BAD
    assert _append(lib, [None] * 8, T_total=0) == kda.KDA_OK
    assert lib.kda_last_launch_count() == 0


def test_outputs_lie_over_no_part_of_another_array(lib):
    """An output that begins or ends inside another array of the call is refused; out
    may be q itself."""
    def pairs(call, sizes, outs, free=()):
        for i in outs:
            for j in range(len(sizes)):
                if i == j or (i, j) in free or (j, i) in free:
                    continue
                for into in (0, sizes[j] - 16, 16 - sizes[i]):
                    if into % 16 == 0 and -sizes[i] < into < sizes[j]:
                        at = [(1 << 24) + (k << 20) for k in range(len(sizes))]
                        at[i] = at[j] + into
                        assert call([V(x) for x in at]) == BAD, (i, j, into)
    pool, scales = 8 * 16 * 2 * 64, 8 * 2 * 4
    # q, k, v, k_scales, v_scales, table, cu, kv, out
    sizes = [8 * 4 * 128, pool, pool, scales, scales, 32, 16, 16, 8 * 4 * 128]
    pairs(lambda p: _attn(lib, p), sizes, (8,), free=((8, 0),))
    # qkv, positions, slots, q, k, v, k_scales, v_scales
    sizes = [8 * 8 * 128, 32, 32, 8 * 4 * 128, pool, pool, scales, scales]
    pairs(lambda p: _append(lib, p), sizes, (3, 4, 5, 6, 7))
    # logits, tokens, logprobs, entropy, ranks, top_ids, top_logprobs
    sizes = [8 * 128 * 4, 32, 32, 32, 32, 8 * 16, 8 * 16]
    pairs(lambda p: _logprobs(lib, p), sizes, (2, 3, 4, 5, 6))
    assert lib.kda_last_launch_count() == 0


def _logprobs(lib, ptrs=None, **kw):
    base = dict(N=8, V=128, n_top=4, dtype=kda.KDA_F32, stride=128, scale=1.0, workspace=WS,
                workspace_bytes=256)
    base.update(kw)
    return lib.kda_token_logprobs(*(ptrs or _at(7)), ctypes.byref(kda.KdaLogprobsArgs(**base)))


@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), BAD), (dict(V=0), BAD), (dict(n_top=-1), BAD), (dict(dtype=2), BAD),
    (dict(stride=127), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(scale=3e38), BAD),
    (dict(scale=2.0 ** 65), BAD), (dict(scale=2.0 ** -65), BAD),
    (dict(V=(1 << 24) + 1, stride=1 << 25), UNSUP), (dict(N=(1 << 20) + 1), UNSUP),
    (dict(n_top=65), UNSUP), (dict(stride=1 << 50), UNSUP), (dict(workspace=None), BAD),
    (dict(workspace_bytes=255), BAD)])
def test_logprobs_refuses(lib, kw, want):
    assert _logprobs(lib, **kw) == want
    assert lib.kda_last_launch_count() == 0


def test_logprobs_refuses_pointers(lib):
    for i in range(7):
        ptrs = _at(7)
        ptrs[i] = V((1 << 24) + 2)
        assert _logprobs(lib, ptrs) == BAD, i
    for i in (0, 1, 5, 6):       # (a log probability and a rank want a token)
        ptrs = _at(7)
        ptrs[i] = None
        assert _logprobs(lib, ptrs) == BAD, i
    assert lib.kda_token_logprobs(*_at(7), None) == BAD
    assert _logprobs(lib, [None] * 7, N=0) == kda.KDA_OK
    assert lib.kda_last_launch_count() == 0


def test_binding_refuses_host_tensors_types_and_shapes():
    kda.build()
    bf, f32, f8, i32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32
    z = lambda *s, dt=bf: torch.zeros(s, dtype=dt)
    ws = z(256, dt=torch.uint8)
    good = dict(q=z(8, 4, 64), k=z(8, 32, 2, 64, dt=f8), v=z(8, 32, 2, 64, dt=f8),
                ks=z(8, 2, 2, dt=f32), vs=z(8, 2, 2, dt=f32), t=z(2, 4, dt=i32), cu=z(3, dt=i32),
                kv=z(2, dt=i32), out=z(8, 4, 64))

    def attn(**kw):
        a = dict(good, **kw)
        kda.kda_paged_attn_q8(a["q"], a["k"], a["v"], a["ks"], a["vs"], a["t"], a["cu"], a["kv"],
                              a["out"], workspace=ws)
    with pytest.raises(ValueError, match="CUDA device"):
        attn()
    for kw, what in ((dict(q=good["q"].half()), TypeError), (dict(k=z(8, 32, 2, 64)), TypeError),
                     (dict(v=z(8, 32, 2, 64, dt=torch.float8_e5m2)), TypeError),
                     (dict(ks=z(8, 2, 2)), TypeError), (dict(vs=z(8, 32, 2, dt=f32)), ValueError),
                     (dict(ks=z(8, 2, 2, dt=f32).transpose(1, 2)), ValueError),
                     (dict(out=z(8, 4, 64, dt=f32)), TypeError)):
        with pytest.raises(what):
            attn(**kw)

    def append(**kw):
        a = dict(qkv=z(8, 8, 64), slot=z(8, dt=i32), q=z(8, 4, 64), **{n: good[n] for n in ("k", "v", "ks", "vs")})
        a.update(kw)
        kda.kda_paged_append_q8(a["qkv"], None, None, None, None, a["slot"], a["q"], a["k"], a["v"],
                                a["ks"], a["vs"], workspace=ws)
    with pytest.raises(ValueError, match="CUDA device"):
        append()
    for kw, what in ((dict(k=z(8, 32, 2, 64)), TypeError), (dict(vs=z(8, 1, 2, dt=f32)), ValueError),
                     (dict(qkv=z(8, 7, 64)), ValueError), (dict(qkv=z(8, 8, 64).half()), TypeError)):
        with pytest.raises(what):
            append(**kw)

    def logprobs(x, t=None, ids=None, top=None, n=3):
        t = z(n, dt=i32) if t is None else t
        kda.kda_token_logprobs(x, t, z(n, dt=f32), None, None, ids, top, workspace=ws)
    with pytest.raises(ValueError, match="CUDA device"):
        logprobs(z(3, 9))
    for a, what in (((z(3, 9).half(),), TypeError), ((z(9),), ValueError),
                    ((z(9, 3).t(),), ValueError), ((z(1, 9).expand(3, 9),), ValueError),
                    ((z(3, 9), z(3, dt=torch.int64)), TypeError),
                    ((z(3, 9), None, z(3, 2, dt=i32)), ValueError),
                    ((z(3, 9), None, z(3, 2, dt=i32), z(3, 1, dt=f32)), ValueError)):
        with pytest.raises(what):
            logprobs(*a)


def test_plain_forms_of_the_scales_and_the_rounding():
    """The tests' own 64-bit forms against the type's conversion and against a search."""
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(4000, generator=g) * torch.exp2(torch.randint(-14, 9, (4000,), generator=g).float()),
                   torch.arange(-448, 449) / 64.0, torch.tensor([0.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9])])
    x = x.clamp(-448, 448)
    assert torch.equal(rounded(x.double()), x.to(torch.float8_e4m3fn).double())
    for a in (0.0, 1e-30, 2.0 ** -60, 447.0, 448.0, 449.0, 3.5, 3.51, 1e30):
        p = float(scale_for(torch.tensor(a, dtype=torch.float64)))
        assert 2.0 ** -50 <= p <= 2.0 ** 50
        assert a <= 448 * p or p == 2.0 ** 50
        assert p == 2.0 ** -50 or a > 448 * p / 2
