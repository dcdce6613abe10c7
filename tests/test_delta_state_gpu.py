"""How exactly the gated delta rule holds its states, by norms: with keys that
are alike, whose T has large entries, as with random ones."""
import pytest
import torch

import delta_reference as ref
import state_space_model_ssm_amd as ssm

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = ref.U


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(L, H, K, V, seed, cosine, strength, rate=0.002):
    """One row; the keys' cosines are about `cosine`, beta is sigmoid(N + strength)."""
    g = torch.Generator().manual_seed(seed)
    unit = torch.nn.functional.normalize
    k = (1 - cosine) ** 0.5 * unit(torch.randn(1, L, 1, K, generator=g), dim=-1) + cosine ** 0.5 * unit(torch.randn(K, generator=g), dim=0)
    q, k = (unit(t, dim=-1).to(BF16) for t in (torch.randn(1, L, 1, K, generator=g), k))
    v = torch.randn(1, L, H, V, generator=g).to(BF16)
    dec = -rate * torch.nn.functional.softplus(torch.randn(1, L, H, generator=g))
    beta = torch.sigmoid(torch.randn(1, L, H, generator=g) + strength)
    return q, k, v, dec, beta, 0.5 * torch.randn(1, H, V, K, generator=g)


def cuda(*ts):
    return [t.cuda() for t in ts]


@pytest.mark.parametrize("cosine,strength", [(0.0, 0.0), (0.5, 3.0), (0.9, 3.0), (0.99, 3.0), (0.9, 0.0)])
@pytest.mark.parametrize("L,H,K,V", [(640, 2, 128, 128), (640, 2, 64, 64), (2500, 1, 64, 128), (2000, 1, 128, 64)])
def test_the_last_state_is_held_to_float32_whatever_the_keys(L, H, K, V, cosine, strength):
    """In one chain and over segments.  Factors in three parts lose 2^-26 a product, float32 sums of up to 128 terms
    2^-24 for each of their roundings, of which 2^1 to 2^3 add up by norms; T's largest row sum, 2 at most for keys that
    are alike, passes on what reaches it: 2^-20, which is less than 1e-6."""
    q, k, v, g, beta, h0 = make(L, H, K, V, L + K, cosine, strength)
    want = ref.gdr(*(ref.f64(t) for t in (q, k, v, g, beta, h0)))[1]
    got = ref.f64(ssm.gdr_fwd(*cuda(q, k, v, g, beta), h0=h0.cuda())[1])
    far = float((got - want).norm() / want.norm())
    print(f"{far:.2e}")
    assert far <= 2.0 ** -20
    # Asked for beside what the backward starts from, too.
    both = ssm.gdr_fwd(*cuda(q, k, v, g, beta), h0=h0.cuda(), return_states=True)[1]
    assert torch.equal(both.cpu().double(), got)


@pytest.mark.parametrize("gates", [F32, BF16])
@pytest.mark.parametrize("L,nqk,K,V", [(200, 4, 64, 64), (333, 2, 128, 128), (130, 1, 128, 64), (1100, 1, 64, 128)])
def test_gradients_of_gates_head_by_head(L, nqk, K, V, gates):
    """Decays of about 1, 3e-1, 7e-3 and 3e-7 a token beside each other: dg has its own decay as a factor, and is held
    to that.  By norms of one head: at most five products in turn of factors in two parts, 3 * 2^-18 each, and its own
    rounding: each value is off by U of itself at most, so their norm by U of theirs.  (1 / sqrt(3) of that holds for
    many values of a size, not for these, a few of which make the norm.)  Where the gate is shut (below -200), dg is 0."""
    q, k, v, g, beta, h0 = make(L, 4, K, V, L + V, 0.0, 0.0)
    gen = torch.Generator().manual_seed(K)
    q, k = (torch.nn.functional.normalize(torch.randn(1, L, nqk, K, generator=gen), dim=-1).to(BF16) for _ in range(2))
    g = (-torch.tensor([0.01, 1.0, 5.0, 15.0]) * (0.8 + 0.4 * torch.rand(1, L, 4, generator=gen))).to(gates)
    g[0, 37, 0], g[0, 70, 1], g[0, 127, 2], g[0, 64, 3] = -float("inf"), -1e30, -300.0, -1000.0
    beta = beta.to(gates)
    dy, dh = torch.randn(1, L, 4, V, generator=gen).to(BF16), torch.randn(1, 4, V, K, generator=gen)
    want = ref.gdr_bwd(*(ref.f64(t) for t in (q, k, v, g.clamp(min=-1e4), beta, dy, h0)), dh_last=ref.f64(dh))[0]
    cs = cuda(q, k, v, g, beta)
    states = ssm.gdr_fwd(*cs, h0=h0.cuda(), return_states=True)[2]
    got = ssm.gdr_bwd(*cs, states, dy.cuda(), dh_last=dh.cuda())
    shut = g[0].float() <= -200
    assert int(shut.sum()) == 4 and not got[3][0].cpu()[shut].any()
    for name, t in (("dg", got[3]), ("dbeta", got[4])):
        for h in range(4):
            w = want[name][0, :, h]
            far = float((ref.f64(t[0, :, h]) - w).norm() / w.norm())
            print(name, h, f"{far:.1e}")
            assert far <= 2.0 ** -14 + (U if gates == BF16 else 0.0), (name, h, far)


@pytest.mark.parametrize("L,K,V", [(1, 64, 64), (150, 128, 128), (200, 64, 128), (3000, 128, 64)])
def test_a_token_whose_beta_is_zero_writes_nothing(L, K, V):
    """Whatever its key and value are: every output and gradient of the others has the same bits."""
    q, k, v, g, beta, h0 = make(L, 2, K, V, L, 0.5, 1.0)
    gen = torch.Generator().manual_seed(V)
    shut = torch.rand(L, generator=gen) < 0.4
    shut[-1] = True
    beta[0, shut] = 0.0
    dy, dh = torch.randn(1, L, 2, V, generator=gen).to(BF16), torch.randn(1, 2, V, K, generator=gen)
    other = [q, k.clone(), v.clone(), g, beta]
    other[1][0, shut] = torch.randn(int(shut.sum()), 1, K, generator=gen).to(BF16)
    other[2][0, shut] = 1e3 * torch.randn(int(shut.sum()), 2, V, generator=gen).to(BF16)
    outs = []
    for args in ((q, k, v, g, beta), other):
        cs = cuda(*args)
        y, last, states = ssm.gdr_fwd(*cs, h0=h0.cuda(), return_states=True)
        dq, dk, dv, dg, dbeta, dh0 = ssm.gdr_bwd(*cs, states, dy.cuda(), dh_last=dh.cuda())
        assert not dv[0, shut.cuda()].any()
        on = ~shut.cuda()
        outs.append((y, last, dq, dk[0, on], dv, dg, dbeta[0, on], dh0))
        if not shut[0] or L == 1:
            want = ref.gdr_bwd(*(ref.f64(t) for t in (*args, dy, h0)), dh_last=ref.f64(dh))[0]["dbeta"]
            # Products of factors in two parts, five in turn at most: 5 * 3 * 2^-18, by norms.
            assert float((ref.f64(dbeta) - want).norm()) <= 2.0 ** -14 * float(want.norm())
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_shut_gates_keep_a_state():
    """No beta and no decay: the state, bit for bit, over many tokens, and nothing from nothing."""
    q, k, v, g, beta, h0 = make(2000, 40, 64, 64, 5, 0.0, 0.0)
    g, beta = torch.zeros_like(g), torch.zeros_like(beta)
    assert torch.equal(ssm.gdr_fwd(*cuda(q, k, v, g, beta), h0=h0.cuda())[1].cpu(), h0)
    y, last = ssm.gdr_fwd(*cuda(q, k, v, g, beta))
    assert not y.any() and not last.any()


@pytest.mark.parametrize("cosine,strength", [(0.0, 0.0), (0.5, 3.0), (0.9, 3.0)])
@pytest.mark.parametrize("L,H,K,V,rate", [(640, 2, 128, 128, 0.01), (640, 2, 64, 64, 0.3), (2500, 1, 64, 128, 0.002), (300, 4, 128, 64, 5.0)])
def test_float32_gradients_by_norms(L, H, K, V, rate, cosine, strength):
    """dg, dbeta and dh0.  A product of two factors in two parts loses 3 * 2^-18 of its terms at most, 2^-18 of them by
    norms, where roundings are spread over their half steps; five in turn, each of which passes the others' on, 2^-15.7
    with T's row sums of 2 at most on two of them: 2^-15 is a third of 1e-4, which a mistaken term would be."""
    q, k, v, g, beta, h0 = make(L, H, K, V, L + K, cosine, strength, rate)
    gen = torch.Generator().manual_seed(L)
    dy, dh = torch.randn(1, L, H, V, generator=gen).to(BF16), torch.randn(1, H, V, K, generator=gen)
    want = ref.gdr_bwd(*(ref.f64(t) for t in (q, k, v, g, beta, dy, h0)), dh_last=ref.f64(dh))[0]
    cs = cuda(q, k, v, g, beta)
    for last in (True, False):
        states = ssm.gdr_fwd(*cs, h0=h0.cuda(), return_h_last=last, return_states=True)[2]
        got = ssm.gdr_bwd(*cs, states, dy.cuda(), dh_last=dh.cuda())
        for name, t in zip(("dg", "dbeta", "dh0"), got[3:]):
            far = float((ref.f64(t) - want[name]).norm() / want[name].norm())
            print(name, f"{far:.1e}")
            assert far <= 2.0 ** -15, (name, far)


@pytest.mark.parametrize("gate", [3, 4])
def test_a_gate_that_is_not_finite_reaches_its_own_head(gate):
    """From the start of its 64 tokens on."""
    args = list(make(200, 3, 64, 64, 3, 0.0, 0.0))[:5]
    clean = ssm.gdr_fwd(*cuda(*args))
    args[gate] = args[gate].clone()
    args[gate][0, 100, 1] = float("nan")
    y, last = ssm.gdr_fwd(*cuda(*args))
    others = [0, 2]
    assert torch.equal(y[0, :64], clean[0][0, :64]) and torch.equal(y[0, :, others], clean[0][0, :, others])
    assert torch.equal(last[0, others], clean[1][0, others])
    assert y[0, 100:, 1].isnan().all() and last[0, 1].isnan().all()
