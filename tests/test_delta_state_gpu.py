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
