"""GPU parity of kda_paged_plan, kda_paged_append and kda_verify_drafts with
plain forms, and a run of a whole serving step (plan, append, attention, draft
verification and the KDA commit that follows it)."""

import pytest
import torch

import hybrid_linear_attention_delta_gb300 as kda
import oracle
from hybrid_linear_attention_delta_gb300 import inputs
from kda_cases import TOL, rel
from paged_cases import (DT, AttnCase, append_reference, half_step, plan_reference,
                         verify_reference)

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.lib()


def _i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


# ------------------------------------------------------------------------ plan

class PlanCase:
    """Requests with shuffled pages and a ring of free ones."""

    def __init__(self, new, cached, held, page, free, head, width=None, pad=0, seed=0):
        g = torch.Generator().manual_seed(seed)
        B = len(new)
        self.page, self.T = page, sum(new) + pad
        n_held = sum(held)
        n_pages = max(1, n_held + free)
        order = torch.randperm(n_pages, generator=g).tolist()
        want = [-(-(n + c) // page) for n, c in zip(new, cached)]
        width = width or max([1] + want + list(held))
        self.table = [[-7] * width for _ in range(B)]
        at = 0
        for b in range(B):
            for j in range(held[b]):
                self.table[b][j] = order[at]
                at += 1
        self.ring = [-9] * n_pages
        self.head, self.count = head % n_pages, free
        for i in range(free):
            self.ring[(self.head + i) % n_pages] = order[n_held + i]
        self.cu = [0]
        for n in new:
            self.cu.append(self.cu[-1] + n)
        self.cached, self.held = list(cached), list(held)

    def run(self, ws=None):
        B = len(self.cached)
        t = dict(cu=_i32(self.cu), cached=_i32(self.cached),
                 table=_i32(self.table).reshape(B, -1) if B else torch.zeros((0, 1), dtype=I32, device="cuda"),
                 held=_i32(self.held), ring=_i32(self.ring), state=_i32([self.head, self.count]),
                 held_out=_i32([-1] * B), ring_out=_i32([-1, -1]), kv=_i32([-1] * B),
                 positions=_i32([-1] * self.T), slots=_i32([-2] * self.T))
        self.ws = ws if ws is not None else kda.paged_workspace_for()
        self.dev = t
        for _ in range(2):   # repeatable: its outputs are not among its inputs
            kda.kda_paged_plan(t["cu"], t["cached"], t["table"], t["held"], t["ring"], t["state"],
                               t["held_out"], t["ring_out"], t["kv"], t["positions"], t["slots"],
                               page_size=self.page, workspace=self.ws)
        return t

    def check(self, bits=0):
        t = self.run()
        assert kda.kda_device_status(self.ws)[1] == bits
        ref = plan_reference(self.cu, self.cached, self.table, self.held, self.ring, self.head,
                             self.count, self.page, self.T)
        for name, want in ref.items():
            got = t[name].cpu().tolist()
            assert got == want, name
        return t


def _random_plan(B, page, top_new, top_cached, seed, free=None, **kw):
    g = torch.Generator().manual_seed(seed)
    r = lambda hi: torch.randint(0, hi + 1, (B,), generator=g).tolist()
    new, cached = r(top_new), r(top_cached)
    held = [-(-c // page) for c in cached]
    for b in range(0, B, 5):      # finished, or rolled back with pages to spare
        if b % 2:
            new[b], cached[b] = 0, 0
        else:
            held[b] += 2
    need = sum(max(0, -(-(n + c) // page) - h) for n, c, h in zip(new, cached, held))
    return PlanCase(new, cached, held, page, need if free is None else free, seed * 37, seed=seed,
                    **kw)


@pytest.mark.parametrize("B,page,top_new,top_cached", [
    (1, 16, 1, 0), (1, 256, 5000, 9000), (7, 16, 1, 200), (64, 64, 8, 5000), (33, 128, 700, 0),
    (512, 16, 3, 300), (513, 32, 60, 100), (1500, 16, 20, 90), (8192, 16, 2, 40)])
def test_plan_matches_request_by_request(B, page, top_new, top_cached):
    _random_plan(B, page, top_new, top_cached, seed=B).check()
    _random_plan(B, page, top_new, top_cached, seed=B + 1, pad=19).check()


def test_plan_without_requests_or_tokens():
    PlanCase([], [], [], 16, 5, 3).check()
    PlanCase([], [], [], 16, 5, 3, pad=40).check()
    PlanCase([0, 0, 0], [0, 31, 0], [0, 2, 4], 16, 5, 3).check()


def test_plan_ring_wraps():
    for head in range(0, 13):
        PlanCase([20, 0, 33], [0, 0, 5], [0, 4, 1], 16, 8, head, seed=head).check()


def test_plan_refuses_what_does_not_fit():
    """Requests in order until the first that does not fit; later ones that need
    pages are refused too, those that need none are served."""
    c = PlanCase([40, 100, 1, 1, 5], [0, 0, 0, 20, 16], [0, 0, 0, 2, 1], 16, 4, 2)
    t = c.check(bits=256)
    assert t["kv"].tolist() == [40, 0, 0, 21, 0]
    c = PlanCase([3, 5, 2], [1, -4, 7], [0, 0, 0], 16, 6, 0)
    assert c.check(bits=128)["kv"].tolist() == [4, 0, 9]
    c = PlanCase([3, 5, 2], [1, 4, 7], [0, 0, 0], 16, 6, 0, width=2)
    c.cached[1], c.held[2] = 28, 9
    assert c.check(bits=128)["kv"].tolist() == [4, 0, 0]


def test_plan_bad_inputs_on_the_device():
    c = PlanCase([3, 5], [10, 4], [1, 1], 16, 6, 1, pad=2)
    c.cu = [0, 9, 8]
    t = c.run()
    assert kda.kda_device_status(c.ws) == (kda.KDA_ERR_DEVICE_CHECK, 4)
    assert t["kv"].tolist() == [0, 0] and (t["slots"] == -1).all()
    assert t["held_out"].tolist() == c.held and t["ring_out"].tolist() == [c.head, c.count]
    assert t["table"].tolist() == c.table and t["ring"].tolist() == c.ring
    # a ring state out of range counts as empty
    c = PlanCase([3, 5], [10, 20], [1, 1], 16, 6, 1)
    c.count = 99
    t = c.run()
    assert kda.kda_device_status(c.ws)[1] == 512 | 256
    assert t["kv"].tolist() == [13, 0]
    # a free page that is no page: its tokens have no slot
    c = PlanCase([3, 5], [10, 20], [1, 1], 16, 6, 1)
    c.ring[c.head] = 1 << 20
    t = c.run()
    assert kda.kda_device_status(c.ws)[1] == 512
    assert t["slots"].tolist()[3:] == [-1] * 5 and min(t["slots"].tolist()[:3]) >= 0
    # a page that is none is given back: it is told
    c = PlanCase([0, 5], [0, 20], [2, 2], 16, 6, 1)
    c.table[0][1] = -3
    t = c.run()
    assert kda.kda_device_status(c.ws)[1] == 512
    assert t["kv"].tolist() == [0, 25] and t["ring_out"].tolist() == [c.head, 8]
    assert t["ring"].tolist()[(c.head + 7) % 10] == -3
    # more pages given back than the ring has room for
    c = PlanCase([0, 0], [0, 0], [3, 3], 16, 2, 1)
    c.count = 5
    t = c.run()
    assert kda.kda_device_status(c.ws)[1] == 512
    assert t["ring_out"].tolist() == [c.head, 8]


def test_plan_token_counts_near_the_end_of_32_bits():
    """The longest batch that T_total can name: positions, slots and padding up to
    row 2^31 - 2, a request whose last rows lie there and whose cache is at its
    longest."""
    page, width = 256, 1 << 22                  # width * page = 2^30
    T = (1 << 31) - 1
    new = [1 << 30, (1 << 30) - 4096, 300]      # ends 3797 rows before T
    cached = [0, 0, (1 << 30) - 300]
    n_pages = (1 << 23) - 1
    cu = [0, new[0], new[0] + new[1], sum(new)]
    table = torch.full((3, width), 5, dtype=I32, device="cuda")
    ring = torch.arange(n_pages, dtype=I32, device="cuda").flip(0).contiguous()
    head = 1000
    held, kv, held_out = _i32([0, 0, width]), _i32([0] * 3), _i32([0] * 3)
    pos = torch.full((T,), -3, dtype=I32, device="cuda")
    slot = torch.full((T,), -3, dtype=I32, device="cuda")
    state = _i32([0, 0])
    ws = kda.paged_workspace_for()

    def plan():
        kda.kda_paged_plan(_i32(cu), _i32(cached), table, held, ring, _i32([head, n_pages]),
                           held_out, state, kv, pos, slot, page_size=page, workspace=ws)
    plan()
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    assert kv.tolist() == [new[0], new[1], 1 << 30]
    first = [0, width, None]
    step = 1 << 27
    for b in range(3):
        for a in range(cu[b], cu[b + 1], step):
            e = min(cu[b + 1], a + step)
            want = cached[b] + torch.arange(a - cu[b], e - cu[b], device="cuda")
            assert torch.equal(pos[a:e].long(), want)
            pages = (n_pages - 1 - (head + first[b] + want // page) % n_pages) if b < 2 else 5
            assert torch.equal(slot[a:e].long(), pages * page + want % page)
    assert (pos[cu[3]:] == 0).all() and (slot[cu[3]:] == -1).all()
    cu[2] = -1                                   # bad: every row is marked
    plan()
    assert kda.kda_device_status(ws) == (kda.KDA_ERR_DEVICE_CHECK, 4)
    assert all((slot[a:a + step] == -1).all() and (pos[a:a + step] == 0).all()
               for a in range(0, T, step))


# ---------------------------------------------------------------------- append

def _append_case(T, Hq, Hkv, d, rot, page, dtype, norm, max_pos, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    n_pages = -(-T // page) + 2
    qkv = (2.0 * torch.randn((T, Hq + 2 * Hkv, d), generator=g)).to(dt)
    wq = 1 + 0.2 * torch.randn(d, generator=g) if norm else None
    wk = 1 + 0.2 * torch.randn(d, generator=g) if norm else None
    rope = kda.rope_table(max_pos, rot, device="cpu") if rot else None
    pos = torch.randint(0, max_pos, (T,), generator=g).to(I32)
    slot = torch.randperm(n_pages * page, generator=g)[:T].to(I32)
    if pad:
        slot[T - pad:] = -1
    return qkv, wq, wk, rope, pos, slot, n_pages


def _append(c, Hq, Hkv, d, page, mode, eps=1e-6):
    qkv, wq, wk, rope, pos, slot, n_pages = c
    dev = lambda x: None if x is None else x.cuda()
    q = torch.full((qkv.shape[0], Hq, d), 5.0, dtype=qkv.dtype, device="cuda")
    k = torch.full((n_pages, page, Hkv, d), 3.0, dtype=qkv.dtype, device="cuda")
    v = torch.full_like(k, 4.0)
    ws = kda.paged_workspace_for()
    kda.kda_paged_append(dev(qkv), dev(wq), dev(wk), dev(rope), dev(pos), dev(slot), q, k, v,
                         rope_mode=mode, norm_eps=eps, workspace=ws)
    return q, k, v, ws


def _check_append(c, Hq, Hkv, d, page, mode, skipped=()):
    qkv, wq, wk, rope, pos, slot, n_pages = c
    q, k, v, ws = _append(c, Hq, Hkv, d, page, mode)
    assert kda.kda_device_status(ws)[1] == (0 if not skipped else skipped)
    live = (slot >= 0) & (slot < n_pages * page)
    if rope is not None:
        live &= (pos >= 0) & (pos < rope.shape[0])
    (rq, sq), (rk, sk), rv = append_reference(qkv, wq, wk, rope, torch.where(live, pos, 0), Hq,
                                              Hkv, mode, 1e-6)
    # one rounding to the type, and in fp32 the d products of the mean (half of
    # their relative error reaches the root), the root, two products of the norm
    # and three operations of the rotation
    def close(got, ref, size):
        fp32 = (d / 2 + 16) * half_step(torch.float32)
        tol = half_step(qkv.dtype) * ref.abs() * 1.01 + fp32 * size + 1e-30
        bad = (got.double().cpu() - ref).abs() > tol
        assert not bad.any(), float((got.double().cpu() - ref).abs().max())
    close(q[live.cuda()], rq[live], sq[live])
    assert (q[(~live).cuda()] == 5.0).all()
    at = slot[live].long().cuda()
    fk, fv = k.view(-1, Hkv, d), v.view(-1, Hkv, d)
    close(fk[at], rk[live], sk[live])
    assert torch.equal(fv[at].cpu(), qkv[live][:, Hq + Hkv:])
    rest = torch.ones(n_pages * page, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (fk[rest] == 3.0).all() and (fv[rest] == 4.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rots", [(64, (0, 16, 32, 64)), (128, (0, 16, 48, 64, 128))])
@pytest.mark.parametrize("mode", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [True, False])
def test_append_rotations_and_norms(dtype, d, rots, mode, norm):
    for rot in rots:
        c = _append_case(37, 6, 2, d, rot, 16, dtype, norm, 5000, seed=rot + d)
        _check_append(c, 6, 2, d, 16, mode)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hkv,d", [(1, 1, 1, 64), (1, 32, 8, 128), (3, 5, 1, 128),
                                        (700, 7, 7, 64), (129, 64, 1, 64), (1000, 32, 8, 128)])
def test_append_shapes(dtype, T, Hq, Hkv, d):
    c = _append_case(T, Hq, Hkv, d, d, 32, dtype, True, 1 << 20, seed=T)
    _check_append(c, Hq, Hkv, d, 32, "half")


def test_append_skips_padding_and_bad_tokens():
    c = _append_case(40, 4, 2, 64, 64, 16, "bf16", True, 100, seed=3, pad=9)
    _check_append(c, 4, 2, 64, 16, "half")
    c[5][3] = c[6] * 16          # a slot behind the pool
    _check_append(c, 4, 2, 64, 16, "half", skipped=1)
    c[4][5], c[4][6] = 100, -1   # positions outside the table
    _check_append(c, 4, 2, 64, 16, "half", skipped=1 | 1024)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", ["half", "interleaved"])
def test_append_beyond_32_bit_offsets(dtype, mode):
    """More than 2^31 elements in the projection, the queries and the pages."""
    T, Hq, Hkv, d, page = 176000, 96, 16, 128, 64
    n_pages = (1 << 31) // (page * Hkv * d) + 300
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(7)
    qkv = torch.zeros((T, Hq + 2 * Hkv, d), dtype=dt, device="cuda")
    rows = torch.cat([torch.arange(64), torch.arange(T // 2, T // 2 + 64), torch.arange(T - 64, T)]).cuda()
    qkv[rows] = torch.randn((192, Hq + 2 * Hkv, d), generator=g, device="cuda").to(dt)
    slot = torch.randperm(n_pages * page, generator=g, device="cuda")[:T].to(I32)
    slot[rows[-64:]] = torch.arange(n_pages * page - 64, n_pages * page, device="cuda").to(I32)
    taken = (slot[:-64] >= n_pages * page - 64).nonzero()[:, 0]
    slot[taken] = -1                      # (slots are distinct)
    pos = torch.arange(T, device="cuda").to(I32)
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    rope = kda.rope_table(T, d)
    q = torch.zeros((T, Hq, d), dtype=dt, device="cuda")
    k, v = (torch.zeros((n_pages, page, Hkv, d), dtype=dt, device="cuda") for _ in range(2))
    ws = kda.paged_workspace_for()
    kda.kda_paged_append(qkv, wq, wk, rope, pos, slot, q, k, v, rope_mode=mode, workspace=ws)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    rows = rows[slot[rows] >= 0]
    (rq, sq), (rk, sk), rv = append_reference(qkv[rows].cpu(), wq.cpu(), wk.cpu(), rope.cpu(),
                                              pos[rows].cpu(), Hq, Hkv, mode, 1e-6)
    at = slot[rows].long()
    for got, ref, size in ((q[rows], rq, sq), (k.view(-1, Hkv, d)[at], rk, sk)):
        tol = half_step(dt) * ref.abs() * 1.01 + (d / 2 + 16) * half_step(torch.float32) * size + 1e-30
        assert ((got.double().cpu() - ref).abs() <= tol).all()
    assert torch.equal(v.view(-1, Hkv, d)[at], qkv[rows][:, Hq + Hkv:])


def test_append_zero_tokens():
    ws = kda.paged_workspace_for()
    e = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    kda.kda_paged_append(e(0, 6, 64), None, None, None, None, _i32([]), e(0, 4, 64),
                         e(1, 16, 1, 64), e(1, 16, 1, 64), workspace=ws)
    assert kda.kda_last_launch_count() == 0


# ---------------------------------------------------------------------- verify

def _verify_case(N, n, V, dtype, seed, noise=0.5, probs=True):
    g = torch.Generator().manual_seed(seed)
    logits = 3 * torch.randn((N, n + 1, V), generator=g)
    p = torch.softmax(logits, -1).to(DT[dtype])
    q = torch.softmax(logits[:, :n] + noise * torch.randn((N, n, V), generator=g), -1)
    x = torch.zeros((N, n), dtype=I32)
    if n:
        x = torch.multinomial(q.flatten(0, 1), 1, generator=g).view(N, n).to(I32)
    q = q.to(DT[dtype])
    return [p, q if probs else None, x, torch.rand((N, n), generator=g),
            torch.rand((N,), generator=g)]


def _verify(c, lens=None):
    p, q, x, ua, us = [None if t is None else t.cuda() for t in c]
    N, n1, _ = p.shape
    acc, tok = _i32([-5] * N), torch.full((N, n1), -5, dtype=I32, device="cuda")
    ws = kda.paged_workspace_for()
    kda.kda_verify_drafts(p, q, x, ua, us, acc, tok,
                          None if lens is None else _i32(lens), workspace=ws)
    return acc.cpu(), tok.cpu(), kda.kda_device_status(ws)[1]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("N,n,V", [(1, 0, 1), (1, 1, 2), (3, 2, 7), (1, 7, 32000), (64, 7, 1000),
                                   (40, 3, 1031), (9, 4, 50257), (2, 1, 131072), (200, 5, 333),
                                   (5, 0, 4099), (1, 40, 512)])
def test_verify_matches_plain_form(dtype, probs, N, n, V):
    for seed in range(3):
        c = _verify_case(N, n, V, dtype, seed=seed * 100 + V, probs=probs,
                         noise=0.1 if seed == 0 else 0.6)
        acc, tok, bits = _verify(c)
        racc, rtok = verify_reference(*c)
        assert bits == 0
        assert torch.equal(acc, racc) and torch.equal(tok, rtok)


# More segments of 1024 tokens to a CTA than a warp has lanes,
# with aligned rows and others; more than it has threads; so many that
# they are longer; the largest vocabulary; the most drafts.
@pytest.mark.parametrize("N,n,V,dtype", [
    (64, 1, 151936, "bf16"), (128, 1, 128256, "f32"), (160, 1, 40009, "bf16"), (160, 1, 600000, "f32"),
    (160, 0, 600001, "bf16"), (8, 1, (1 << 23) + 5, "f32"), (160, 1, 5000000, "bf16"),
    (154, 0, 4194305, "f32"), (2, 1, 1 << 24, "f32"), (1, 1024, 257, "f32"), (3, 1000, 5000, "bf16")])
@pytest.mark.parametrize("probs", [True, False])
def test_verify_sizes_up_to_the_limits(probs, N, n, V, dtype):
    g = torch.Generator(device="cuda").manual_seed(V + n)
    dt = DT[dtype]
    p = torch.empty((N, n + 1, V), dtype=dt, device="cuda")
    q = torch.empty((N, n, V), dtype=dt, device="cuda")
    x = torch.zeros((N, n), dtype=I32, device="cuda")
    for i in range(N):
        logits = 3 * torch.randn((n + 1, V), generator=g, device="cuda")
        p[i] = torch.softmax(logits, -1).to(dt)
        # few of the drafts stand, or nearly all of them where there are many
        noise = 0.02 if n > 8 else 0.6
        q[i] = torch.softmax(logits[:n] + noise * torch.randn((n, V), generator=g, device="cuda"), -1).to(dt)
        if n:
            x[i] = torch.multinomial(q[i].float(), 1, generator=g)[:, 0].to(I32)
    ua = torch.rand((N, n), generator=g, device="cuda") * (0.2 if n > 8 else 1.0)
    c = [p, q if probs else None, x, ua, torch.rand((N,), generator=g, device="cuda")]
    acc, tok, bits = _verify(c)
    racc, rtok = verify_reference(*c)
    assert bits == 0
    assert torch.equal(acc, racc) and torch.equal(tok, rtok)


def test_verify_ragged_drafts():
    c = _verify_case(12, 5, 900, "f32", seed=1, noise=0.1)
    lens = [0, 1, 2, 3, 4, 5, 5, 4, 3, 2, 1, 0]
    acc, tok, bits = _verify(c, lens)
    racc, rtok = verify_reference(*c, lens=lens)
    assert bits == 0 and torch.equal(acc, racc) and torch.equal(tok, rtok)
    assert all(a <= 1 + l for a, l in zip(acc.tolist(), lens))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_verify_borders(dtype):
    """u at 0 and just below 1; drafts that match the target exactly (nothing is
    left of p - q: the draw is from p); one-token distributions."""
    p, q, x, ua, us = _verify_case(6, 3, 2000, dtype, seed=8)
    us[0], us[1] = 0.0, 1.0 - 2.0 ** -24
    q[2:4] = p[2:4, :3]
    ua[2:4] = 1.0 - 2.0 ** -24
    x[3, 1] = 11
    p[3, 1, 11] = q[3, 1, 11] = 0       # 0 < 0: this draft does not stand
    p[4] = 0
    p[4, :, 1999] = 1.0                 # all mass on the last token
    p[5] = 0
    p[5, :, 0] = 1.0
    c = [p, q, x, ua, us]
    acc, tok, bits = _verify(c)
    racc, rtok = verify_reference(*c)
    assert bits == 0 and torch.equal(acc, racc) and torch.equal(tok, rtok)
    assert acc[2] == 4 and acc[3] == 2


def test_verify_far_tokens_are_not_lost():
    """One heavy token and a long tail: the tail's borders lie within the
    rounding of an fp32 sum, and every draw still has to find its token."""
    V = 120001
    tail = torch.full((V,), 0.5 / (V - 1), dtype=torch.float32)
    tail[17] = 0.5
    N = 64
    p = tail.expand(N, 1, V).contiguous()
    us = torch.rand((N,), generator=torch.Generator().manual_seed(2))
    c = [p, None, torch.zeros((N, 0), dtype=I32), torch.zeros((N, 0)), us]
    acc, tok, bits = _verify(c)
    racc, rtok = verify_reference(*c)
    assert bits == 0 and torch.equal(acc, racc) and torch.equal(tok, rtok)


@pytest.mark.parametrize("N,V", [(3, 16 * 1024 + 1), (19, 33 * 1024), (19, 65 * 1024 - 3),
                                 (1, 73 * 1024), (76, 65 * 1024 + 8), (152, 17000)])
@pytest.mark.parametrize("probs", [True, False])
def test_verify_sequences_on_several_ctas(probs, N, V):
    """Two, four and eight CTAs a sequence, the last of them with few segments (it
    has its sum long before the others), launch after launch; sequences with a bad
    length between them, whose CTAs leave at once."""
    c = _verify_case(N, 2, V, "bf16", seed=V, probs=probs)
    lens = [(-1 if n % 5 == 2 else n % 3) for n in range(N)]
    good = [n for n in range(N) if lens[n] >= 0]
    pick = lambda t: None if t is None else t[good]
    racc, rtok = verify_reference(*(pick(t) for t in c), lens=[lens[n] for n in good])
    for _ in range(8):
        acc, tok, bits = _verify(c, lens)
        assert bits == (128 if len(good) < N else 0)
        assert torch.equal(acc[good], racc) and torch.equal(tok[good], rtok)
        bad = torch.ones(N, dtype=torch.bool)
        bad[good] = False
        assert (acc[bad] == 0).all() and (tok[bad] == -1).all()


# Four rows, found by search: the mass of segments 0, 2, ... 30 of 1024 tokens, that
# of segment 40, and u, for which u times the sum lies between two values that
# sums in different orders give the border behind a segment with mass.
GAPS = [
    (16, "0x1.b0a24ep-1", "0x1.07cbeap-2",
     "0x1.c13056p-1 0x1.d602ap-2 0x1.e2c394p-1 0x1.5f382cp-13 0x1.43a47cp-5 0x1.031cacp-2 "
     "0x1.bea34ap-18 0x1.7167b4p-9 0x1.f0c782p-24 0x1.74fc3cp-5 0x1.a0d156p-6 "
     "0x1.58fdeep-6 0x1.96894ep-19 0x1.f5f8cap-4 0x1.0beea4p-14 0x1.3778fcp-14"),
    (20, "0x1.4c4b14p-1", "0x1.30c7ccp+0",
     "0x1.b0790cp-1 0x1.dbd38p-11 0x1.c92292p-16 0x1.5179cep-7 0x1.71fb98p-19 "
     "0x1.e560d2p-4 0x1.54b324p-2 0x1.ef3a5ap-24 0x1.067714p-14 0x1.c9e13p-1 0x1.7151ecp-9 "
     "0x1.142b9cp-17 0x1.2a259ap-12 0x1.49f1dep-10 0x1.a8f24ap-23 0x1.9a34a2p-19"),
    (22, "0x1.f3f3a2p-1", "0x1.358824p-4",
     "0x1.d0629ep-1 0x1.f7410cp-1 0x1.db59ecp-13 0x1.69015p-8 0x1.1946ep-16 0x1.1a5edp-8 "
     "0x1.64aceep-23 0x1.6ac5e2p-1 0x1.6a6194p-5 0x1.a9e0a6p-17 0x1.5ce42ep-1 "
     "0x1.c845bcp-1 0x1.ef19a6p-8 0x1.db0904p-10 0x1.1420c6p-6 0x1.3720dp-15"),
    (30, "0x1.70a224p-1", "0x1.d84e8ep-1",
     "0x1.ba60a2p-14 0x1.232738p-8 0x1.5db0b4p-8 0x1.26c9d6p-19 0x1.96e8a2p-17 "
     "0x1.eae3bp-21 0x1.eb71acp-1 0x1.f941f8p-16 0x1.d365fcp-4 0x1.d2371cp-21 "
     "0x1.fc6992p-24 0x1.11fdbcp-23 0x1.14bfa2p-1 0x1.b358ecp-15 0x1.7ea80cp-1 "
     "0x1.4b6b6ap-14"),
]


def test_verify_border_between_two_roundings():
    """The draw finds a token with mass although the place that it seeks falls on
    a border whose two roundings enclose it, with segments without mass behind."""
    V, N = 65536, 160
    p, us = torch.zeros((N, 1, V)), torch.zeros((N,))
    for n in range(N):
        _, u, last, m = GAPS[n % len(GAPS)]
        p[n, 0, 5:32 * 1024:2048] = torch.tensor([float.fromhex(x) / 4 for x in m.split()])
        p[n, 0, 40 * 1024 + 5] = float.fromhex(last) / 4
        us[n] = float.fromhex(u)
    acc, tok, bits = _verify([p, None, torch.zeros((N, 0), dtype=I32), torch.zeros((N, 0)), us])
    assert bits == 0 and (acc == 1).all()
    for n in range(N):
        seg = GAPS[n % len(GAPS)][0]  # either side of the border is a fair draw
        assert tok[n, 0] in (seg * 1024 + 5, (seg + 2 if seg < 30 else 40) * 1024 + 5)


def test_verify_bad_inputs_on_the_device():
    p, q, x, ua, us = _verify_case(4, 2, 300, "f32", seed=4, noise=0.0)
    x[0, 0], x[1, 1] = 300, -1
    acc, tok, bits = _verify([p, q, x, ua, us])
    racc, rtok = verify_reference(p, q, x, ua, us)
    assert bits == 2048 and torch.equal(acc, racc) and torch.equal(tok, rtok)
    assert acc[0] == 1
    acc, tok, bits = _verify([p, q, x, ua, us], lens=[0, 3, -1, 0])
    assert bits == 128 and acc.tolist() == [1, 0, 0, 1]
    assert (tok[1:3] == -1).all()
    p[2] = 0.0
    p[3, 0] = float("nan")
    acc, tok, bits = _verify([p, q, x, ua, us], lens=[0, 0, 0, 0])
    assert bits == 4096 and tok[2, 0] == -1 and tok[3, 0] == -1


def test_arrays_side_by_side_in_one_buffer():
    """A plan and a verification whose arrays touch each other in one allocation."""
    c = PlanCase([20, 0, 33, 1], [0, 0, 5, 16], [0, 4, 1, 1], 16, 8, 3, seed=2)
    B, width, n_pages, T = 4, len(c.table[0]), len(c.ring), c.T
    ref = plan_reference(c.cu, c.cached, c.table, c.held, c.ring, c.head, c.count, c.page, T)
    fill = dict(cu=c.cu, cached=c.cached, table=sum(c.table, []), held=c.held, ring=c.ring,
                state=[c.head, c.count], held_out=[-1] * B, ring_out=[-1, -1], kv=[-1] * B,
                positions=[-1] * T, slots=[-2] * T)
    buf, t, at = _i32(sum(fill.values(), [])), {}, 0
    for name, x in fill.items():
        t[name] = buf[at:at + len(x)]
        at += len(x)
    t["table"] = t["table"].view(B, width)
    ws = kda.paged_workspace_for()
    kda.kda_paged_plan(*t.values(), page_size=c.page, workspace=ws)
    assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
    for name, want in ref.items():
        assert t[name].tolist() == want, name
    c = _verify_case(5, 3, 700, "f32", seed=3)
    x, lens, acc = c[2], [3, 0, 2, 1, 3], [0] * 5
    buf = _i32(x.flatten().tolist() + lens + acc + [0] * 20)
    draft, n_draft, accepted, tokens = buf[:15].view(5, 3), buf[15:20], buf[20:25], buf[25:].view(5, 4)
    kda.kda_verify_drafts(c[0].cuda(), c[1].cuda(), draft, c[3].cuda(), c[4].cuda(), accepted, tokens,
                          n_draft, workspace=ws)
    racc, rtok = verify_reference(*c, lens=lens)
    assert torch.equal(accepted.cpu(), racc) and torch.equal(tokens.cpu(), rtok)


# ------------------------------------------------------------------- a whole step

def test_serving_steps_together():
    """Speculative serving over several steps: plan, append and attention on the
    paged side, verification of the drafts, and the KDA layer's verify-and-commit
    fed by what was accepted.  The pages end up holding exactly the accepted
    history, the attention sees it, and the KDA state is the recurrence over it."""
    torch.manual_seed(0)
    B, Hq, Hkv, d, page, n, V, H = 3, 4, 2, 64, 16, 3, 500, 2
    n_tok = n + 1
    n_pages, width = 24, 8
    dt = torch.bfloat16
    g = torch.Generator().manual_seed(1)
    k_pages = torch.full((n_pages, page, Hkv, d), float("nan"), dtype=dt, device="cuda")
    v_pages = torch.full_like(k_pages, float("nan"))
    table = torch.zeros((B, width), dtype=I32, device="cuda")
    held, ring = [_i32([0] * B), _i32([0] * B)], _i32(list(range(n_pages)))
    state = [_i32([5, n_pages]), _i32([0, 0])]
    cached = _i32([0] * B)
    T = B * n_tok
    cu = _i32([n_tok * b for b in range(B + 1)])
    kv, pos, slot = _i32([0] * B), _i32([0] * T), _i32([0] * T)
    rope = kda.rope_table(256, d)
    w = torch.ones(d, device="cuda")
    ws = kda.paged_workspace_for(T, Hq, Hkv, d)
    kws = kda.workspace_for(B, H, B)
    pool = inputs.pool_states(B, H, 128, 128, 7).cuda()
    start = pool.cpu().clone()
    slots = _i32(list(range(B)))
    kept = [[] for _ in range(B)]             # the KDA layer's accepted tokens, per request
    history = [[] for _ in range(B)]          # (k, v) rows of accepted tokens, per request
    prev = accepted = None
    for step in range(6):
        qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=g).to(dt).cuda()
        q, out = (torch.zeros((T, Hq, d), dtype=dt, device="cuda") for _ in range(2))
        a, b = step % 2, 1 - step % 2
        kda.kda_paged_plan(cu, cached, table, held[a], ring, state[a], held[b], state[b], kv, pos,
                           slot, page_size=page, workspace=ws)
        kda.kda_paged_append(qkv, w, w, rope, pos, slot, q, k_pages, v_pages, workspace=ws)
        kda.kda_paged_attn(q, k_pages, v_pages, table, cu, kv, out, workspace=ws)
        tt = {m: t.cuda() for m, t in inputs.token_tensors(T, H, 128, 128, dt, 50 + step).items()}
        ko = torch.empty_like(tt["v"])
        kda.kda_decode_spec(tt["q"], tt["k"], tt["v"], tt["g"], tt["beta"], slots, pool, ko, n_tok,
                            *((prev[m] for m in ("k", "v", "g", "beta")) if prev else (None,) * 4),
                            accepted, n_tok if prev else 0, workspace=kws)
        c = _verify_case(B, n, V, "f32", seed=step, noise=0.4)
        accepted, tokens = _i32([0] * B), torch.zeros((B, n_tok), dtype=I32, device="cuda")
        kda.kda_verify_drafts(*[t.cuda() for t in c], accepted, tokens, workspace=ws)
        racc, rtok = verify_reference(*c)
        assert torch.equal(accepted.cpu(), racc) and torch.equal(tokens.cpu(), rtok)
        assert kda.kda_device_status(ws) == (kda.KDA_OK, 0)
        assert kda.kda_device_status(kws) == (kda.KDA_OK, 0)
        # the attention against a plain one over the accepted history and this step's tokens
        kf, vf = k_pages.view(-1, Hkv, d).cpu(), v_pages.view(-1, Hkv, d).cpu()
        for r in range(B):
            rows = slice(r * n_tok, (r + 1) * n_tok)
            here = [(kf[s], vf[s]) for s in slot[rows].long().tolist()]
            K = torch.stack([x[0] for x in history[r] + here])
            Vv = torch.stack([x[1] for x in history[r] + here])
            total = len(history[r]) + n_tok
            assert int(kv[r]) == total
            one = AttnCase([n_tok], [total], Hq=Hq, Hkv=Hkv, d=d, page=total, dtype="bf16",
                           extra_pages=0)
            one.k[:], one.v[:], one.q = K, Vv, q[rows].cpu()
            ref, size, top = one.reference()
            assert ((out[rows].double().cpu() - ref).abs() <= one.bound(ref, size, top)).all()
            history[r] += here[:int(racc[r])]
            kept[r] += [(step, r * n_tok + j) for j in range(int(racc[r]))]
        cached = cached + accepted
        prev = tt
    # the last step's commit: the pool holds the recurrence over the accepted tokens
    kda.kda_decode_spec(None, None, None, None, None, slots, pool, None, 0, prev["k"], prev["v"],
                        prev["g"], prev["beta"], accepted, n_tok, workspace=kws)
    assert kda.kda_device_status(kws) == (kda.KDA_OK, 0)
    drawn = [inputs.token_tensors(T, H, 128, 128, dt, 50 + step) for step in range(6)]
    for r in range(B):
        seq = {m: torch.stack([drawn[s][m][i] for s, i in kept[r]]) for m in drawn[0]}
        _, want, _ = oracle.decode_pool(seq["q"], seq["k"], seq["v"], seq["g"], seq["beta"], [r],
                                        start, len(kept[r]), False)
        assert rel(pool[r], want[r]) <= TOL["bf16"]
    # all requests finish: every page is free again, each exactly once
    cached, cu0 = _i32([0] * B), _i32([0] * (B + 1))
    a, b = 0, 1
    kda.kda_paged_plan(cu0, cached, table, held[a], ring, state[a], held[b], state[b], kv,
                       pos[:0], slot[:0], page_size=page, workspace=ws)
    head, count = state[b].tolist()
    assert count == n_pages and sorted(ring.tolist()) == list(range(n_pages))
    assert held[b].tolist() == [0] * B
