"""CPU-side checks of the paged full-attention and draft-verification calls:
host-visible argument errors return before any launch, workspace sizes, and the
binding's refusals."""

import ctypes

import pytest
import torch

import hybrid_linear_attention_delta_gb300 as kda

V = ctypes.c_void_p
FAKE = V(4096)   # never dereferenced: every case fails a host check first
WS = V(1 << 20)
BAD, UNSUP = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    kda.build()
    return kda.lib()


def _args(**kw):
    base = dict(B=2, T_total=8, Hq=4, Hkv=2, d=64, page_size=16, n_pages=8, max_pages=4,
                dtype=kda.KDA_BF16, workspace=WS, workspace_bytes=1 << 30)
    base.update(kw)
    return kda.KdaPagedArgs(**base)


def _attn(lib, a, ptrs=None, scale=0.1, causal=1):
    return lib.kda_paged_attn(*(ptrs or [FAKE] * 7), scale, causal, ctypes.byref(a))


def test_workspace_grows_with_the_batch_up_to_a_bound(lib):
    f = kda.kda_paged_workspace_bytes
    assert f(0, 4, 2, 64) % 256 == 0 and f(0, 4, 2, 64) > 0
    assert f(1, 8, 1, 128) <= f(64, 8, 1, 128) <= f(4096, 8, 1, 128) == f(1 << 20, 8, 1, 128)
    assert f(1 << 20, 8, 1, 128) <= 42 << 20
    assert f(5, 4, 3, 64) == 0          # heads that do not divide


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=7), BAD), (dict(Hq=0), BAD), (dict(Hkv=0), BAD), (dict(Hq=5), BAD),
    (dict(d=96), UNSUP), (dict(d=256), UNSUP), (dict(Hq=130, Hkv=2), UNSUP),
    (dict(page_size=0), BAD), (dict(page_size=48), UNSUP), (dict(page_size=8), UNSUP),
    (dict(page_size=512), UNSUP), (dict(n_pages=0), BAD), (dict(n_pages=1 << 27), UNSUP),
    (dict(max_pages=0), BAD), (dict(max_pages=1 << 27), UNSUP),
    (dict(max_pages=(1 << 26) + 1), UNSUP), (dict(B=-1), BAD),
    (dict(B=8193), UNSUP), (dict(T_total=-1), BAD), (dict(workspace=None), BAD),
    (dict(workspace=V(1 << 20 | 16)), BAD), (dict(workspace_bytes=4096), BAD)])
def test_attention_refuses(lib, kw, want):
    assert _attn(lib, _args(**kw)) == want
    assert lib.kda_last_launch_count() == 0


def test_attention_refuses_pointers_and_scalars(lib):
    for i in range(7):
        for p in (None, V(4098)):
            ptrs = [FAKE] * 7
            ptrs[i] = p
            assert _attn(lib, _args(), ptrs) == BAD
    assert _attn(lib, _args(), scale=float("nan")) == BAD
    assert _attn(lib, _args(), scale=float("inf")) == BAD
    assert _attn(lib, _args(), causal=2) == BAD
    assert lib.kda_paged_attn(*([FAKE] * 7), 0.1, 1, None) == BAD
    # nothing to do: no launch, no pointer looked at
    assert _attn(lib, _args(B=0), [None] * 7) == kda.KDA_OK
    assert _attn(lib, _args(T_total=0), [None] * 7) == kda.KDA_OK
    assert lib.kda_last_launch_count() == 0


def test_plan_refuses(lib):
    call = lambda a, ptrs=None: lib.kda_paged_plan(
        *(ptrs or [V(4096 + 256 * i) for i in range(11)]), None if a is None else ctypes.byref(a))
    assert call(None) == BAD
    for kw, want in ((dict(page_size=20), UNSUP), (dict(n_pages=-1), BAD), (dict(max_pages=0), BAD),
                     (dict(B=-2), BAD), (dict(B=9000), UNSUP), (dict(workspace=None), BAD),
                     (dict(workspace_bytes=128), BAD)):
        assert call(_args(**kw)) == want
    for i in range(11):
        for p in (None, V(4097)):
            ptrs = [V(4096 + 256 * j) for j in range(11)]
            ptrs[i] = p
            assert call(_args(), ptrs) == BAD
    ptrs = [V(4096 + 256 * j) for j in range(11)]
    ptrs[6] = ptrs[3]                    # held_out over held
    assert call(_args(), ptrs) == BAD
    ptrs = [V(4096 + 256 * j) for j in range(11)]
    ptrs[7] = ptrs[5]                    # ring_out over ring
    assert call(_args(), ptrs) == BAD
    assert lib.kda_last_launch_count() == 0


def test_append_refuses(lib):
    def call(a=None, f=None, ptrs=None):
        base = dict(q_norm=FAKE, k_norm=FAKE, rope=FAKE, max_pos=10, rot_dim=32, rope_mode=0,
                    norm_eps=1e-6)
        base.update(f or {})
        return lib.kda_paged_append(*(ptrs or [FAKE] * 6),
                                    ctypes.byref(kda.KdaAppendArgs(**base)),
                                    ctypes.byref(_args(**(a or {}))))
    for kw, want in ((dict(dtype=3), BAD), (dict(d=32), UNSUP), (dict(page_size=24), UNSUP),
                     (dict(T_total=-1), BAD), (dict(workspace=None), BAD)):
        assert call(a=kw) == want
    for kw, want in ((dict(rot_dim=-16), BAD), (dict(rot_dim=80), BAD), (dict(rot_dim=24), UNSUP),
                     (dict(rope=None), BAD), (dict(max_pos=0), BAD), (dict(rope_mode=2), BAD),
                     (dict(norm_eps=-1.0), BAD), (dict(norm_eps=float("nan")), BAD),
                     (dict(q_norm=V(4100)), BAD), (dict(rope=V(4100)), BAD)):
        assert call(f=kw) == want
    for i in range(6):
        for p in (None, V(4098)):
            ptrs = [FAKE] * 6
            ptrs[i] = p
            assert call(ptrs=ptrs) == BAD
    assert lib.kda_paged_append(*([FAKE] * 6), None, ctypes.byref(_args())) == BAD
    assert call(a=dict(T_total=0), ptrs=[None] * 6) == kda.KDA_OK
    assert lib.kda_last_launch_count() == 0


def test_verify_refuses(lib):
    def call(ptrs=None, **kw):
        base = dict(N=2, n_draft=3, V=100, dtype=kda.KDA_F32, workspace=WS, workspace_bytes=256)
        base.update(kw)
        return lib.kda_verify_drafts(*(ptrs or [FAKE] * 8),
                                     ctypes.byref(kda.KdaVerifyArgs(**base)))
    for kw, want in ((dict(N=-1), BAD), (dict(n_draft=-1), BAD), (dict(V=0), BAD),
                     (dict(dtype=2), BAD), (dict(n_draft=1025), UNSUP),
                     (dict(V=(1 << 24) + 1), UNSUP), (dict(N=(1 << 20) + 1), UNSUP),
                     (dict(workspace=None), BAD), (dict(workspace_bytes=255), BAD)):
        assert call(**kw) == want
    for i in (0, 2, 4, 5, 6, 7):
        ptrs = [FAKE] * 8
        ptrs[i] = None
        assert call(ptrs) == BAD
    for i in range(8):
        ptrs = [FAKE] * 8
        ptrs[i] = V(4097)
        assert call(ptrs) == BAD
    assert lib.kda_verify_drafts(*([FAKE] * 8), None) == BAD
    assert call([None] * 8, N=0) == kda.KDA_OK
    assert lib.kda_last_launch_count() == 0


def test_outputs_are_arrays_of_their_own(lib):
    """CTAs read inputs at different times: an output over another array is
    refused before a launch."""
    ptr = lambda n: [V(4096 + 4096 * i) for i in range(n)]

    def pairs(call, n, outs, others):
        for i in outs:
            for j in list(outs) + list(others):
                if i != j:
                    ptrs = ptr(n)
                    ptrs[i] = ptrs[j]
                    assert call(ptrs) == BAD, (i, j)

    a = _args()
    # block_table, free_ring, held_out, ring_out, kv_lens, positions, slot_map
    pairs(lambda p: lib.kda_paged_plan(*p, ctypes.byref(a)), 11, (2, 4, 6, 7, 8, 9, 10),
          (0, 1, 3, 5))
    pairs(lambda p: _attn(lib, a, p), 7, (6,), (1, 2))
    f = kda.KdaAppendArgs(None, None, FAKE, 10, 32, 0, 1e-6)
    pairs(lambda p: lib.kda_paged_append(*p, ctypes.byref(f), ctypes.byref(a)), 6, (3, 4, 5), (0,))
    v = kda.KdaVerifyArgs(2, 3, 100, kda.KDA_F32, None, WS, 256)
    pairs(lambda p: lib.kda_verify_drafts(*p, ctypes.byref(v)), 8, (6, 7), (2, 3))
    assert lib.kda_last_launch_count() == 0


def test_attention_refuses_scales_that_overflow_in_powers_of_two(lib):
    for scale in (2.4e38, -3.4e38):
        assert _attn(lib, _args(), [V((1 << 24) + (k << 20)) for k in range(7)], scale=scale) == BAD
    assert lib.kda_last_launch_count() == 0


def test_outputs_lie_over_no_part_of_another_array(lib):
    """An output that begins or ends inside another array of the call, or inside the
    workspace, is refused like one at its address."""
    def pairs(call, sizes, outs, free=()):
        # arrays of `sizes` bytes, 2^20 apart from address 2^24 on; the last is the workspace
        for i in outs:
            for j in range(len(sizes)):
                if i == j or (i, j) in free or (j, i) in free:
                    continue
                for into in (0, sizes[j] - 16, 16 - sizes[i]):
                    if into % 16 == 0 and -sizes[i] < into < sizes[j] and call.aligned(i, into):
                        at = [(1 << 24) + (k << 20) for k in range(len(sizes))]
                        at[i] = at[j] + into
                        assert call([V(x) for x in at]) == BAD, (i, j, into)

    class Call:
        def __init__(self, fn, n):
            self.fn, self.n = fn, n

        def __call__(self, at):
            return self.fn(at[:-1], at[-1])

        def aligned(self, i, into):     # the workspace stays where it may lie
            return i != self.n or into % 256 == 0

    def plan(p, ws):
        return lib.kda_paged_plan(*p, ctypes.byref(_args(B=8, T_total=64, n_pages=64, max_pages=8,
                                                         workspace=ws)))
    # cu, cached, table, held, ring, state, held_out, state_out, kv, positions, slots
    pairs(Call(plan, 11), [48, 32, 256, 32, 256, 16, 32, 16, 32, 256, 256, 256],
          (2, 4, 6, 7, 8, 9, 10, 11))

    def attn(p, ws):
        return lib.kda_paged_attn(*p, 0.1, 1, ctypes.byref(_args(workspace=ws)))
    # q, k, v, table, cu, kv, out
    sizes = [8 * 4 * 128, 8 * 16 * 2 * 128, 8 * 16 * 2 * 128, 32, 16, 16, 8 * 4 * 128, 1 << 16]
    pairs(Call(attn, 7), sizes, (6, 7), free=((6, 0),))
    p = [V((1 << 24) + (k << 20)) for k in range(7)]
    for into in (16, 8 * 4 * 128 - 16, -16):      # out may be q, but not lie across it
        p[6] = V((1 << 24) + into)
        assert attn(p, V(1 << 20)) == BAD

    def append(p, ws):
        f = kda.KdaAppendArgs(p[6], p[7], p[8], 16, 32, 0, 1e-6)
        return lib.kda_paged_append(*p[:6], ctypes.byref(f), ctypes.byref(_args(workspace=ws)))
    # qkv, positions, slots, q, k, v, q_norm, k_norm, rope
    pairs(Call(append, 9), [8 * 8 * 128, 32, 32, 8 * 4 * 128, 8 * 16 * 2 * 128, 8 * 16 * 2 * 128,
                            256, 256, 2048, 256], (3, 4, 5, 9))

    def verify(p, ws):
        a = kda.KdaVerifyArgs(8, 3, 128, kda.KDA_F32, None, ws, 256)
        return lib.kda_verify_drafts(*p, ctypes.byref(a))
    # p, q, drafts, lens, u_accept, u_sample, accepted, tokens
    pairs(Call(verify, 8), [8 * 4 * 512, 8 * 3 * 512, 96, 32, 96, 32, 32, 128, 256], (6, 7, 8))
    assert lib.kda_last_launch_count() == 0


def test_binding_refuses_host_tensors_types_and_shapes():
    """Tensors off the GPU never reach the library (it would read them there)."""
    kda.build()
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    good = dict(q=z(8, 4, 64), k=z(8, 16, 2, 64), v=z(8, 16, 2, 64), t=i(2, 4), cu=i(3), kv=i(2),
                out=z(8, 4, 64))

    def attn(**kw):
        a = dict(good, **kw)
        kda.kda_paged_attn(a["q"], a["k"], a["v"], a["t"], a["cu"], a["kv"], a["out"],
                           workspace=ws)
    with pytest.raises(ValueError, match="CUDA device"):
        attn()
    with pytest.raises(TypeError):
        attn(q=good["q"].half())
    with pytest.raises(TypeError):
        attn(k=good["k"].float())
    with pytest.raises(ValueError):
        attn(k=z(8, 16, 64))
    with pytest.raises((ValueError, TypeError)):
        attn(t=good["t"].long())
    with pytest.raises(ValueError):
        kda.kda_verify_drafts(z(2, 4, 9, dt=torch.float32), None, i(2, 3), torch.zeros(2, 3),
                              torch.zeros(2), i(2), i(2, 4), workspace=ws)
    with pytest.raises(ValueError):
        kda.rope_table(0, 16, device="cpu")


def test_rope_table_angles_of_far_positions():
    """cos and sin of position 10^6 to fp32, where an fp32 angle is off by 0.06."""
    t = kda.rope_table(1_000_001, 16, device="cpu")[1_000_000].double()
    i = torch.arange(8, dtype=torch.float64)
    a = 1_000_000.0 * 10000.0 ** (-i / 8)
    ref = torch.cat([torch.cos(a), torch.sin(a)])
    assert float((t - ref).abs().max()) <= 2.0 ** -24
