"""The gated delta rule (forward, backward, step) against float64."""
import pytest
import torch

import delta_reference as ref
import state_space_model_ssm_amd as ssm

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = ref.U
# Errors besides y's own rounding, relative to the sizes of what is summed.  A
# float32 factor in two bfloat16 parts is held to 2^-18, and a product of two
# such leaves out another 2^-18: at most 3 * 2^-18 each for the four products
# from one chunk's state to the next and to y (keys with the state, T, the
# state's update, the attention), with 2^-19 for sums of 128 float32 terms.  T's
# own size (at most a few units for unit keys) is in the factor 2 left over.
SMALL = 2.0 ** -13


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(B, L, nqk, H, K, V, seed, gates=F32, rate=(0.001, 1.0)):
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.nn.functional.normalize(torch.randn(B, L, nqk, K, generator=g), dim=-1).to(BF16) for _ in range(2))
    v = torch.randn(B, L, H, V, generator=g).to(BF16)
    rates = torch.logspace(*(torch.tensor(rate).log10().tolist()), H)
    dec = (-rates * torch.nn.functional.softplus(torch.randn(B, L, H, generator=g))).to(gates)
    beta = torch.sigmoid(torch.randn(B, L, H, generator=g)).to(gates)
    h0 = 0.5 * torch.randn(B, H, V, K, generator=g)
    dy = torch.randn(B, L, H, V, generator=g).to(BF16)
    return q, k, v, dec, beta, h0, dy


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def nan(shape, dtype=F32):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def one_tensor(*parts):
    """The parts as views of one tensor, side by side, as a fused projection leaves them."""
    flat = torch.cat([p.flatten(-2) for p in parts], -1).cuda()
    at, views = 0, []
    for p in parts:
        n = p.shape[-2] * p.shape[-1]
        views.append(flat[..., at:at + n].unflatten(-1, p.shape[-2:]))
        at += n
    return views


def state_tol(states, last):
    """SMALL of the largest state that a row and head goes through (and of values of about 4 that enter it)."""
    return SMALL * max([float(s.abs().max()) for row in states for s in row] + [float(last.abs().max()), 4.0])


def unpack(saved, B, H, chunks, K, V):
    """The states (B, H, chunks, V, K) that a forward saved: two bfloat16 parts, [16 key elements][32 values][part], a lane
    per (element, group g) with the values 4 g .. and 16 + 4 g .."""
    per = saved.view(B, H, chunks, -1)[..., :4 * K * V].contiguous()
    x = per.view(BF16).double().view(B, H, chunks, K // 16, V // 32, 2, 4, 16, 2, 4).sum(5)   # part; g, element, half, value
    return x.permute(0, 1, 2, 4, 7, 5, 8, 3, 6).reshape(B, H, chunks, V, K)


CASES = [  # batch, L, qk heads, value heads, K, V, gates, h0, lengths
    (1, 1, 1, 1, 64, 64, F32, True, None), (2, 2, 1, 2, 128, 64, BF16, False, None),
    (1, 15, 2, 2, 64, 128, F32, True, None), (1, 16, 1, 1, 128, 128, BF16, True, None),
    (2, 17, 2, 4, 64, 64, F32, False, None), (1, 63, 1, 4, 128, 128, F32, True, None),
    (1, 64, 1, 2, 64, 64, F32, True, None), (2, 65, 1, 1, 128, 64, BF16, True, None),
    (1, 127, 2, 2, 128, 128, F32, False, None), (1, 128, 1, 3, 64, 128, F32, True, None),
    (3, 129, 2, 2, 128, 128, BF16, True, [129, 0, 64]), (4, 200, 1, 2, 64, 64, F32, True, [1, 63, 65, 300]),
    (2, 257, 3, 3, 64, 128, F32, False, [-5, 193]), (1, 513, 1, 1, 128, 128, F32, True, None),
    (5, 70, 16, 16, 64, 64, BF16, True, [70, 69, 2, 64, 33]),
    # Long rows of few heads: cut into segments along time, some of which a row does not reach.
    (1, 1500, 1, 2, 64, 64, F32, True, None), (4, 2113, 1, 1, 128, 128, F32, True, [2113, 700, 0, 1537]),
    (1, 2048, 1, 1, 64, 128, BF16, False, None), (2, 3001, 1, 2, 128, 64, F32, False, [64, 2990]),
]


@pytest.mark.parametrize("B,L,nqk,H,K,V,gates,with_h0,lengths", CASES)
def test_forward(B, L, nqk, H, K, V, gates, with_h0, lengths):
    q, k, v, g, beta, h0, _ = make(B, L, nqk, H, K, V, L * 7 + H, gates)
    h0 = h0 if with_h0 else None
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    want, last, states, size = ref.gdr(*(ref.f64(t) for t in (q, k, v, g, beta, h0)), lens)
    if lengths is not None:   # rows behind a length may hold anything
        for b, n in enumerate(lengths):
            for t in (q, k, v, g, beta):
                t[b, max(n, 0):] = float("nan")
    cq, ck, cv = one_tensor(q, k, v)
    cg, cb, ch = cuda(g, beta, h0)
    chunks = -(-L // 64)
    y, hl = nan((B, L, H, V), BF16), nan((B, H, V, K))
    st = torch.full((B * H * chunks * (4 * V * (K + 64) + 26624),), 0xff, dtype=torch.uint8, device="cuda")   # NaN
    got = ssm.gdr_fwd(cq, ck, cv, cg, cb, h0=ch, lengths=None if lens is None else lens.cuda(), return_states=True, y=y,
                      h_last=hl, states=st)
    assert got[0] is y and got[1] is hl and got[2] is st
    tol = state_tol(states, last)
    ref.close(hl, last, tol, "h_last")
    saved = unpack(st, B, H, chunks, K, V)
    for b, row in enumerate(states):
        for c, s in enumerate(row):
            ref.close(saved[b, :, c], s, tol, f"state {c} of row {b}")
        assert saved[b, :, len(row):].isnan().all()   # not written
    ref.close(y, want, U * want.abs() + SMALL * (size + K ** -0.5), "y")
    again = ssm.gdr_fwd(cq, ck, cv, cg, cb, h0=ch, lengths=None if lens is None else lens.cuda())
    assert torch.equal(again[0], y) and torch.equal(again[1], hl)
    if with_h0:   # h_last in the place of h0
        ssm.gdr_fwd(cq, ck, cv, cg, cb, h0=ch, lengths=None if lens is None else lens.cuda(), h_last=ch, y=y)
        assert torch.equal(ch, hl) and torch.equal(y, again[0])


@pytest.mark.parametrize("L,H,K,V", [(700, 2, 128, 128), (640, 1, 64, 64), (2500, 1, 64, 128), (2000, 1, 128, 64)])
def test_the_last_state_is_held_to_float32(L, H, K, V):
    """By norms, in one chain and over segments.  What is left of the roundings to bfloat16 is that of T - I's entries in
    two parts, 2^-18 of each at most and 1 / sqrt(3) of that over many, on the half or less of U that they make (keys of
    unit length, random: entries of K K^T of K^-1/2): 2^-19.8.  Sums of 64 to 128 float32 terms: 2^-22."""
    q, k, v, g, beta, h0, _ = make(1, L, 1, H, K, V, L + K, rate=(0.001, 0.02))
    want = ref.gdr(*(ref.f64(t) for t in (q, k, v, g, beta, h0)))[1]
    got = ref.f64(ssm.gdr_fwd(*cuda(q, k, v, g, beta), h0=h0.cuda())[1])
    assert float((got - want).norm()) <= 2.0 ** -19 * float(want.norm())


def by_norm(t):
    """How far an output may be off by norms: 2^-12 and its own rounding.  A rounding is off by at most half a step, U of
    the value, so a few values by that together; over many the errors spread over the half step, and the root of
    their mean square is 1 / sqrt(3) of it at most (the integral of x^2 over 0 .. 1)."""
    return 2.0 ** -12 + (0.0 if t.dtype != BF16 else U if t.numel() < 1024 else U / 3 ** 0.5)


BACKWARD = CASES + [(1, 300, 2, 8, 64, 128, BF16, True, None), (2, 140, 1, 4, 128, 64, F32, True, [140, 77]),
                    # Few heads: time in segments, of rows that end in any of them.
                    (1, 1300, 1, 2, 128, 64, F32, True, None), (2, 1500, 1, 1, 64, 128, BF16, True, [1500, 200]),
                    (3, 1400, 1, 1, 128, 128, F32, False, [1, 0, 1400]), (4, 1024, 2, 2, 64, 64, F32, True, [1024, 129, 128, 900])]


@pytest.mark.parametrize("B,L,nqk,H,K,V,gates,with_h0,lengths", BACKWARD)
def test_backward(B, L, nqk, H, K, V, gates, with_h0, lengths):
    q, k, v, g, beta, h0, dy = make(B, L, nqk, H, K, V, L * 3 + H, gates)
    h0 = h0 if with_h0 else None
    dh = torch.randn(B, H, V, K, generator=torch.Generator().manual_seed(L)) if with_h0 else None
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    want, size = ref.gdr_bwd(*(ref.f64(t) for t in (q, k, v, g, beta, dy, h0)), lens, dh_last=ref.f64(dh))
    if lengths is not None:
        for b, n in enumerate(lengths):
            for t in (q, k, v, g, beta, dy):
                t[b, max(n, 0):] = float("nan")
    cl = None if lens is None else lens.cuda()
    views = one_tensor(q, k, v)
    cg, cb, ch, cdy, cdh = cuda(g, beta, h0, dy, dh)
    states = torch.full((B * H * -(-L // 64) * (4 * V * (K + 64) + 26624),), 0xff, dtype=torch.uint8, device="cuda")   # NaN
    ssm.gdr_fwd(*views, cg, cb, h0=ch, lengths=cl, states=states)
    outs = {n: nan(t.shape, t.dtype) for n, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta))}
    outs["dh0"] = nan((B, H, V, K))
    got = ssm.gdr_bwd(*views, cg, cb, states, cdy, dh_last=cdh, lengths=cl, out=outs)
    names = ("dq", "dk", "dv", "dg", "dbeta", "dh0")
    assert all(t is outs[n] for n, t in zip(names, got))
    for n, t in zip(names, got):
        w = want[n]
        # Five products in turn at most: 5 * 3 * 2^-18 of the sizes, a share of them by norms; heads that share add up.
        if n == "dh0":
            small = 2.0 ** -14 * max(float(w.abs().max()), 4.0 * (1 if dh is None else float(dh.abs().max())))
        else:
            small = 2.0 ** -14 * size[n]
            if n in ("dq", "dk"):
                small = small.unflatten(2, (nqk, -1)).sum(3)
            if n in ("dq", "dk", "dv"):
                small = small[..., None]
        ref.close(t, w, (U * w.abs() if t.dtype == BF16 else 0.0) + small, n)
        far = float((ref.f64(t) - w).norm())
        assert far <= by_norm(t) * float(w.norm()), (n, far / float(w.norm()))
    again = ssm.gdr_bwd(*views, cg, cb, states, cdy, dh_last=cdh, lengths=cl)
    assert all(torch.equal(a, b) for a, b in zip(again, got))


def test_backward_against_differences():
    q, k, v, g, beta, h0, dy = make(1, 70, 1, 2, 64, 64, 12)
    dh = torch.randn(h0.shape, generator=torch.Generator().manual_seed(1))
    states = ssm.gdr_fwd(*cuda(q, k, v, g, beta), h0=h0.cuda(), return_states=True)[2]
    got = ssm.gdr_bwd(*cuda(q, k, v, g, beta), states, dy.cuda(), dh_last=dh.cuda())
    at = [ref.f64(t) for t in (q, k, v, g, beta, h0)]

    def loss(q, k, v, g, beta, h0):
        y, last, _, _ = ref.gdr(q, k, v, g, beta, h0)
        return float((y * dy.double()).sum() + (last * dh.double()).sum())

    eps = 1e-5
    for n, t in enumerate(got):
        for j in torch.randint(t.numel(), (5,), generator=torch.Generator().manual_seed(n)).tolist():
            up, down = [x.clone() for x in at], [x.clone() for x in at]
            up[n].view(-1)[j] += eps
            down[n].view(-1)[j] -= eps
            # Central differences of a float64 loss of order 10^2: 1e-14 / eps, and eps^2 of third derivatives.
            want = (loss(*up) - loss(*down)) / (2 * eps)
            assert abs(float(t.view(-1)[j]) - want) <= U * abs(want) + 2.0 ** -11 * float(t.abs().max()), (n, j)


def test_gradients_of_shut_gates_and_strong_decays():
    """beta of exactly 0 has a gradient, and decays of exp(-200) and less leave the others as they are."""
    q, k, v, g, beta, h0, dy = make(1, 130, 1, 2, 64, 64, 14)
    beta[0, 3], beta[0, 40:44], beta[0, 129] = 0.0, 0.0, 0.0
    g[0, 50], g[0, 100, 1] = -float("inf"), -1000.0
    wide = [ref.f64(t) for t in (q, k, v, g.clamp(min=-1e4), beta, dy, h0)]
    want, size = ref.gdr_bwd(*wide)
    states = ssm.gdr_fwd(*cuda(q, k, v, g, beta), h0=h0.cuda(), return_states=True)[2]
    got = ssm.gdr_bwd(*cuda(q, k, v, g, beta), states, dy.cuda())
    for n, t in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got):
        far = float((ref.f64(t) - want[n]).norm())
        assert far <= by_norm(t) * float(want[n].norm()) + 1e-30, n
    assert got[4][0, 40:44].abs().min() > 0


@pytest.mark.parametrize("B,nqk,H,K,V,gates", [(1, 1, 1, 64, 64, F32), (3, 2, 4, 128, 64, BF16), (2, 1, 3, 64, 128, BF16),
                                               (64, 16, 32, 128, 128, F32), (5, 4, 4, 128, 128, F32)])
def test_step(B, nqk, H, K, V, gates):
    q, k, v, g, beta, h0, _ = make(B, 1, nqk, H, K, V, 3, gates)
    want, last, _, size = ref.gdr(*(ref.f64(t) for t in (q, k, v, g, beta, h0)), scale=0.3)
    views = [t[:, 0] for t in one_tensor(q, k, v)]
    cg, cb, ch = cuda(g[:, 0].contiguous(), beta[:, 0].contiguous(), h0)
    out = nan(h0.shape)
    y, h = ssm.gdr_step(*views, cg, cb, ch, scale=0.3, h_out=out)
    assert h is out and torch.equal(ch.cpu(), h0)
    # float32 throughout: 2^-19 of the terms for sums of 128.
    ref.close(h, last, 2.0 ** -19 * 8, "h")
    ref.close(y, want[:, 0], U * want[:, 0].abs() + 2.0 ** -19 * (size[:, 0] + 4), "y")
    y2, h2 = ssm.gdr_step(*views, cg, cb, ch, scale=0.3)
    assert h2 is ch and torch.equal(h2, out) and torch.equal(y, y2)


def test_steps_continue_a_prompt():
    q, k, v, g, beta, h0, _ = cuda(*make(2, 150, 2, 4, 128, 128, 8))
    whole, last = ssm.gdr_fwd(q, k, v, g, beta, h0=h0)
    y, h = ssm.gdr_fwd(*(t[:, :100] for t in (q, k, v)), g[:, :100].contiguous(), beta[:, :100].contiguous(), h0=h0)
    assert torch.equal(y[:, :64], whole[:, :64])
    for t in range(100, 150):
        yt, h = ssm.gdr_step(*(x[:, t] for x in (q, k, v)), g[:, t].contiguous(), beta[:, t].contiguous(), h)
        # Both are within SMALL of sizes of order 1, and one rounding each.
        assert (yt.float() - whole[:, t].float()).abs().max() <= 2 * U * whole[:, t].float().abs().max() + 2 * SMALL
    assert (h - last).abs().max() <= 2 * SMALL * 4


def test_strong_decays_and_shut_gates():
    """A token that forgets everything (-inf and far below -200), weak ones after it, and betas of 0, 1 and 2."""
    q, k, v, g, beta, h0, _ = make(1, 130, 1, 3, 64, 64, 4)
    g[0, 40], g[0, 70, 0], g[0, 71, 1] = -float("inf"), -1e30, -500.0
    beta[0, 5:9], beta[0, 20], beta[0, 90] = 0.0, 1.0, 2.0
    want, last, states, size = ref.gdr(*(ref.f64(t) for t in (q, k, v, g.clamp(min=-1e4), beta, h0)))
    y, h = ssm.gdr_fwd(*cuda(q, k, v, g, beta), h0=h0.cuda())
    ref.close(h, last, state_tol(states, last), "h")
    ref.close(y, want, U * want.abs() + SMALL * (size + 1), "y")


def test_values_that_are_not_finite_reach_what_is_documented():
    """An infinity in one value channel: that channel, from the start of its 64 tokens on."""
    q, k, v, g, beta, _, _ = make(1, 200, 1, 2, 64, 64, 6)
    clean = ssm.gdr_fwd(*cuda(q, k, v, g, beta))[0]
    v[0, 100, 1, 7] = float("inf")
    y = ssm.gdr_fwd(*cuda(q, k, v, g, beta))[0]
    assert torch.equal(y[0, :64], clean[0, :64]) and torch.equal(y[0, :, 0], clean[0, :, 0])
    others = [c for c in range(64) if c != 7]
    assert torch.equal(y[0, :, 1, others], clean[0, :, 1, others]) and not y[0, 100:, 1, 7].isfinite().any()
