"""Attention steps over an 8-bit ring cache, and its fill, against float64."""
import pytest
import torch

import delta_reference as ref
import state_space_model_ssm_amd as ssm

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = ref.U
SMALL = 2.0 ** -14   # float32 sums and exponentials, weights in two parts (2^-16): of the values' sizes


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(B, L, H, KV, d, seed):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(B, L, H, d, generator=g) * 2).to(BF16)
    # Blocks and heads of unlike sizes, so that a wrong scale shows.
    size = torch.exp(torch.randn(B, -(-L // 16), KV, 1, generator=g)).repeat_interleave(16, 1)[:, :L]
    k, v = ((torch.randn(B, L, KV, d, generator=g) * size).to(BF16) for _ in range(2))
    return q, k, v


def empty(B, KV, window, d, sinks):
    """A cache whose places hold NaN (bytes 0x7f): none may be seen before it is stored."""
    c = ssm.swa_q8_cache(B, KV, window, d, sinks=sinks)
    for t in c:
        t.view(torch.uint8).fill_(0x7f) if t.dtype == torch.float8_e4m3fn else t.fill_(float("nan"))
    return c


def answer(q, cache, b, pos, scale):
    """y of row b at pos and a bound of what its terms add up to."""
    k, v = cache.held(b, 0, pos), cache.held(b, 1, pos)
    H, KV = q.shape[0], k.shape[1]
    k, v = (t.repeat_interleave(H // KV, 1) for t in (k, v))
    p = torch.softmax(torch.einsum("hd,jhd->hj", q.double(), k) * scale, 1)
    return torch.einsum("hj,jhd->hd", p, v), torch.einsum("hj,jhd->hd", p, v.abs())


def check(y, q, model, b, pos, what, scale):
    want, size = answer(q, model, b, pos, scale)
    # The scores' float32 error: 2^-19 of |q||k| summed, at most 2^6 in size here, times the values' sizes.
    ref.close(y, want, U * want.abs() + (SMALL + 2.0 ** -13) * size, what)


@pytest.mark.parametrize("B,H,KV,d,window,sinks,steps", [
    (1, 1, 1, 64, 64, 0, 200), (2, 4, 2, 128, 128, 4, 330), (1, 8, 1, 64, 192, 70, 300), (1, 40, 1, 128, 64, 1, 140),
    (3, 2, 2, 128, 64, 16, 150)])
def test_steps_from_nothing(B, H, KV, d, window, sinks, steps):
    """Token by token from an empty cache, past the window; every row at its own pace."""
    q, k, v = make(B, steps, H, KV, d, steps)
    cache, model = empty(B, KV, window, d, sinks), ref.Q8Cache(B, KV, window, d, sinks)
    cq, ck, cv = q.cuda(), k.cuda(), v.cuda()
    scale = d ** -0.5
    for t in range(steps):
        # Row b starts b steps late, and has no token before.
        pos = torch.tensor([t - 3 * b for b in range(B)], dtype=torch.int32)
        y = ssm.swa_q8_step(cq[:, t], ck[:, t], cv[:, t], cache, pos.cuda(), sinks=sinks)
        for b in range(B):
            p = int(pos[b])
            if p < 0:
                assert not y[b].any()
                continue
            model.rows[b][0].append(k[b, t])
            model.rows[b][1].append(v[b, t])
            if t % 7 == 0 or (p - sinks) % 64 in (62, 63, 0, 1) or p < 3:
                check(y[b], q[b, t], model, b, p, f"row {b} at {p}", scale)


@pytest.mark.parametrize("B,H,KV,d,window,sinks,L,lengths", [
    (1, 2, 1, 128, 64, 0, 64, None), (2, 4, 2, 64, 128, 4, 1, None), (2, 4, 4, 128, 128, 4, 500, [500, 131]),
    (4, 2, 1, 64, 192, 16, 300, [300, 15, 16, 80]), (3, 2, 2, 128, 64, 3, 200, [0, 67, 66])])
def test_fill_then_step(B, H, KV, d, window, sinks, L, lengths):
    q, k, v = make(B, L + 2, H, KV, d, L)
    cache, model = empty(B, KV, window, d, sinks), ref.Q8Cache(B, KV, window, d, sinks)
    lens = [L] * B if lengths is None else lengths
    ssm.swa_q8_fill(k[:, :L].cuda(), v[:, :L].cuda(), cache, sinks=sinks,
                    lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    # The same cache, bit for bit, as the tokens one by one would have left.
    other = empty(B, KV, window, d, sinks)
    for t in range(max(lens)):
        pos = torch.tensor([t if t < n else -1 for n in lens], dtype=torch.int32, device="cuda")
        ssm.swa_q8_step(q[:, t].cuda(), k[:, t].cuda(), v[:, t].cuda(), other, pos, sinks=sinks)
    for b, n in enumerate(lens):
        behind = max(0, n - sinks)
        near = min(n, sinks) if n < sinks else sinks + behind % 64
        whole = min(behind // 64, window // 64)
        assert torch.equal(cache.k_near[b, :, :near], other.k_near[b, :, :near])
        assert torch.equal(cache.v_near[b, :, :near], other.v_near[b, :, :near])
        for x, z in zip(cache[2:], other[2:]):
            m = whole if x.dim() == 3 else whole * 64
            a, c = x[b, :, :m], z[b, :, :m]
            assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))
            rest = x[b, :, m:]
            assert (rest.view(torch.uint8) == 0x7f).all() if x.dim() == 4 else rest.isnan().all()   # left as it was
        for t in range(n):
            model.rows[b][0].append(k[b, t])
            model.rows[b][1].append(v[b, t])
    for step in range(2):
        pos = torch.tensor([n + step for n in lens], dtype=torch.int32)
        rows = torch.arange(B)
        y = ssm.swa_q8_step(*(x[rows, pos.long()].cuda() for x in (q, k, v)), cache, pos.cuda(), sinks=sinks)
        for b in range(B):
            model.rows[b][0].append(k[b, pos[b]])
            model.rows[b][1].append(v[b, pos[b]])
            check(y[b], q[b, pos[b]], model, b, int(pos[b]), f"row {b} step {step}", d ** -0.5)


@pytest.mark.parametrize("B,H,KV,d,window,sinks,L", [(70, 4, 4, 128, 128, 4, 150), (70, 8, 4, 64, 128, 0, 140),
                                                     (66, 4, 4, 64, 1024, 3, 1100)])
def test_many_rows(B, H, KV, d, window, sinks, L):
    """More rows than compute units, which take fewer wavefronts each; prompts of any length, then a token, checked in every fifth row."""
    q, k, v = make(B, L + 1, H, KV, d, L + d)
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32)
    lens[5] = L
    cache, model = empty(B, KV, window, d, sinks), ref.Q8Cache(B, KV, window, d, sinks)
    ssm.swa_q8_fill(k[:, :L].cuda(), v[:, :L].cuda(), cache, sinks=sinks, lengths=lens.cuda())
    rows = torch.arange(B)
    y = ssm.swa_q8_step(*(x[rows, lens.long()].cuda() for x in (q, k, v)), cache, lens.cuda(), sinks=sinks)
    assert not y.isnan().any()
    for b in range(0, B, 5):
        n = int(lens[b])
        model.rows[b][0].extend(k[b, :n + 1])
        model.rows[b][1].extend(v[b, :n + 1])
        check(y[b], q[b, n], model, b, n, f"row {b}", d ** -0.5)


def test_blocks_hold_their_values():
    """Bytes and scales of a whole block: the nearest e4m3 value, ties to even; zeros; a tiny, a huge and a NaN block."""
    B, KV, d, window = 1, 6, 64, 64
    g = torch.Generator().manual_seed(2)
    k = torch.randn(B, 64, KV, d, generator=g).to(BF16)
    k[0, :, 1], k[0, :, 2], k[0, :, 3] = 0.0, k[0, :, 2] * 1e-38, k[0, :, 3] * 1e36
    k[0, 5, 4, 7] = float("nan")
    k[0, 9, 5, 3] = -float("inf")
    cache = empty(B, KV, window, d, 0)
    ssm.swa_q8_fill(k.cuda(), k.cuda(), cache)
    x = k[0].float().transpose(0, 1)
    scale = x.abs().amax((1, 2)) / 448
    got = cache.k_scale[0, :, 0].cpu()
    assert torch.equal(got[:4], scale[:4]) and got[1] == 0 and not got[4:].isfinite().any()
    for c in range(4):
        s = scale[c] if scale[c] > 0 else 1.0
        assert torch.equal(cache.k_ring[0, c].float().cpu().double(), ref.to_e4m3((x[c] / s).clamp(-448, 448).double())), c
    for c in (4, 5):
        values = cache.k_ring[0, c].float().cpu() * cache.k_scale[0, c, 0].cpu()
        assert not values.isfinite().any()
    assert torch.equal(cache.k_ring.view(torch.uint8), cache.v_ring.view(torch.uint8))


def test_the_same_position_again():
    """A step repeated at the same position gives the same cache and the same y; also one that completes a block."""
    q, k, v = (t.cuda() for t in make(2, 200, 4, 2, 128, 7))
    cache = empty(2, 2, 128, 128, 4)
    ssm.swa_q8_fill(k[:, :195], v[:, :195], cache, sinks=4)
    pos = torch.tensor([195, 195], dtype=torch.int32, device="cuda")   # 4 + 3 * 64 - 1: the last of its block
    y = ssm.swa_q8_step(q[:, 195], k[:, 195], v[:, 195], cache, pos, sinks=4)
    kept = [t.clone() for t in cache]
    again = ssm.swa_q8_step(q[:, 195], k[:, 195], v[:, 195], cache, pos, sinks=4)
    assert torch.equal(y, again) and all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(kept, cache))


def test_long_windows_and_far_positions():
    """Windows that several workgroups share, rows anywhere in them, against the bfloat16 cache's attention on the
    values that the 8-bit cache stands for."""
    B, H, KV, d, window, sinks = 5, 16, 4, 128, 4096, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.tensor([5, 700, 4099, 123456, (1 << 30) + 1234], dtype=torch.int32, device="cuda")
    q = torch.randn(B, H, d, generator=g, device="cuda").to(BF16)
    k, v = (torch.randn(B, KV, d, generator=g, device="cuda").to(BF16) for _ in range(2))
    cache = ssm.swa_q8_cache(B, KV, window, d, sinks=sinks)
    for t in cache[:2]:
        t.normal_(generator=g)
    for t in cache[2:4]:
        t.copy_((torch.randn(t.shape, generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn))
    for t in cache[4:]:
        t.copy_(2.0 ** -7 * (1 + torch.rand(t.shape, generator=g, device="cuda")))
    old = [t.clone() for t in cache]
    y = ssm.swa_q8_step(q, k, v, cache, pos, sinks=sinks)
    for b in range(B):
        p = int(pos[b])
        off, now = (p - sinks) % 64, (p - sinks) // 64
        keys, values = [], []
        for t, new, out in ((0, k, keys), (1, v, values)):
            near = old[t][b].clone()
            near[:, sinks + off] = new[b]
            ring = (old[2 + t][b].float().double() * old[4 + t][b].double().repeat_interleave(64, 1)[..., None])
            at = torch.arange(window, device="cuda")
            blk, place = at // 64, at % 64
            # The block there: the last whole one of its number's remainder, or what the token's own block left of it.
            block = blk + (now - blk).div(window // 64, rounding_mode="floor") * (window // 64)
            ok = torch.where(block == now, (place > off) & (now >= window // 64), block >= 0)
            out.append(torch.cat([near[:, :sinks + off + 1].double(), ring[:, ok]], 1))
        for h in range(H):
            s = keys[0][h // 4] @ q[b, h].double() * d ** -0.5
            w = torch.softmax(s, 0)
            want, size = w @ values[0][h // 4], w @ values[0][h // 4].abs()
            ref.close(y[b, h], want.cpu(), (U * want.abs() + (SMALL + 2.0 ** -13) * size).cpu(), (b, h))
