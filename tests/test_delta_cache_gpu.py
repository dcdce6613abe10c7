"""Attention steps over an 8-bit cache at the ends of what they take: tiny
values, any scale of the scores, groups of many heads over split windows."""
import pytest
import torch

import delta_reference as ref
import state_space_model_ssm_amd as ssm

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = ref.U
SMALL = 2.0 ** -14 + 2.0 ** -13   # of the values' sizes: weights in two parts, sums; scores of 2^6 at most, held to 2^-19 of that


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(B, L, H, KV, d, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(B, L, n, d, generator=g).to(BF16) for n in (H, KV, KV)]


def filled(k, v, window, sinks, lengths):
    """A cache and its model after a prompt, and the places that no position owns NaN."""
    B, L, KV, d = k.shape
    cache, model = ssm.swa_q8_cache(B, KV, window, d, sinks=sinks), ref.Q8Cache(B, KV, window, d, sinks)
    for t in cache:
        t.view(torch.uint8).fill_(0x7f) if t.dtype == torch.float8_e4m3fn else t.fill_(float("nan"))
    ssm.swa_q8_fill(k.cuda(), v.cuda(), cache, sinks=sinks, lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    for b, n in enumerate(lengths):
        model.rows[b][0].extend(k[b, :n])
        model.rows[b][1].extend(v[b, :n])
    return cache, model


def answer(q, model, b, pos, scale):
    k, v = (model.held(b, t, pos).repeat_interleave(q.shape[0] // model.rows[b][0][0].shape[0], 1) for t in (0, 1))
    p = torch.softmax((k * q.double()).sum(-1) * scale, 0)[..., None]
    return (p * v).sum(0), (p * v.abs()).sum(0)


def check_step(q, k, v, cache, model, window, sinks, lengths, scale=None):
    """The step at each row's length: y, and the cache that it leaves, against a fill of one token more."""
    B, _, _, d = q.shape
    rows = torch.arange(B)
    pos = torch.tensor(lengths, dtype=torch.int32)
    y = ssm.swa_q8_step(*(t[rows, pos.long()].cuda() for t in (q, k, v)), cache, pos.cuda(), sinks=sinks, scale=scale)
    scale = d ** -0.5 if scale is None else scale
    for b, n in enumerate(lengths):
        model.rows[b][0].append(k[b, n])
        model.rows[b][1].append(v[b, n])
        want, size = answer(q[b, n], model, b, n, scale)
        ref.close(y[b], want, U * want.abs() + SMALL * max(1.0, abs(scale) * d ** 0.5) * size, f"row {b} at {n}")
    after, _ = filled(k, v, window, sinks, [n + 1 for n in lengths])
    for b, n in enumerate(lengths):
        behind = max(0, n + 1 - sinks)
        near, whole = min(n + 1, sinks) if n < sinks else sinks + behind % 64, min(behind // 64, window // 64)
        for x, z in zip(cache[:2], after[:2]):
            assert torch.equal(x[b, :, :near], z[b, :, :near])
        for x, z in zip(cache[2:], after[2:]):
            m = whole * (64 if x.dim() == 4 else 1)
            assert torch.equal(x[b, :, :m].view(torch.uint8), z[b, :, :m].view(torch.uint8))


@pytest.mark.parametrize("size", [1e-22, 1e-26, 1e-30])
@pytest.mark.parametrize("H,KV,d,window", [(4, 2, 64, 128), (2, 1, 128, 1024)])
def test_tiny_values(H, KV, d, window, size):
    """y is as right as of others: the products' least numbers are 2^-126, blocks of 1e-30 have scales of 2^-108."""
    lengths = [window + 75, 40 + 64]
    q, k, v = make(2, window + 76, H, KV, d, d)
    v = (v.float() * size).to(BF16)
    cache, model = filled(k, v, window, 0, lengths)
    check_step(q, k, v, cache, model, window, 0, lengths)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
@pytest.mark.parametrize("H,KV,d,window,sinks", [(4, 2, 64, 128, 4), (6, 2, 128, 1024, 0)])
def test_any_scale(H, KV, d, window, sinks, scale):
    """Negative ones turn the queries round; 0 weighs all that is seen alike."""
    lengths = [sinks + window + 64 + 63, sinks + 2 * window + 10, 70, 3]
    q, k, v = make(4, max(lengths) + 1, H, KV, d, window)
    cache, model = filled(k, v, window, sinks, lengths)
    check_step(q, k, v, cache, model, window, sinks, lengths, scale)


@pytest.mark.parametrize("H,KV,d", [(40, 1, 128), (17, 1, 64), (64, 2, 64)])
def test_many_heads_of_a_key_head_over_split_windows(H, KV, d):
    """Blocks of 16 heads of which each stores the token, and shares of the window that a second kernel joins; at a
    block's last place, its first, and within it, before and after the ring is full."""
    window, sinks = 4096, 3
    lengths = [sinks + 4096 + 64 * 3 - 1, sinks + 1000, sinks + 5000, 1, sinks + 63]
    dims = ssm.SwaDims(batch=5, seqlen=1, nheads=H, nkv=KV, headdim=d, window=window, sinks=sinks, q_batch=H * d, q_token=H * d,
                       k_batch=KV * d, k_token=KV * d, v_batch=KV * d, v_token=KV * d, scale=1.0)
    assert ssm.swa_q8_step_workspace_size(dims) > 0   # it is split
    q, k, v = make(5, max(lengths) + 1, H, KV, d, H)
    cache, model = filled(k, v, window, sinks, lengths)
    check_step(q, k, v, cache, model, window, sinks, lengths)
