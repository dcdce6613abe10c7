"""Norms of queries and keys with the rotation by position, against float64."""
import pytest
import torch

import delta_reference as ref
import state_space_model_ssm_amd as ssm

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = ref.U
# Float32 sums of 256 squares, a root, four products and the sine and cosine: 16 roundings of 2^-24 of the largest
# value's size (a rotation mixes two), and 2^-21 for the reduced angle's float32 fraction of a turn.
SMALL = 2.0 ** -19


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(B, L, H, KV, d, rot, dtype, seed, start=0, weights=True):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(B, L, H + 2 * KV, d, generator=g) * 3).to(dtype)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)) if weights else None for _ in range(2))
    inv = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))).float() if rot else None
    pos = (start + torch.arange(L, dtype=torch.int64) + 1000 * torch.arange(B)[:, None]).to(torch.int32)
    dq, dk = torch.randn(B, L, H, d, generator=g).to(dtype), torch.randn(B, L, KV, d, generator=g).to(dtype)
    return qkv, wq, wk, inv, pos, dq, dk


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def nan(shape, dtype=F32):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


CASES = [  # batch, L, heads, kv heads, headdim, rot, neighbours, dtype, first position, weights
    (1, 1, 1, 1, 16, 16, False, F32, 0, True), (2, 3, 3, 1, 16, 0, False, BF16, 0, True),
    (3, 5, 4, 2, 64, 64, False, BF16, 7, True), (1, 17, 2, 2, 64, 32, True, F32, 1 << 20, True),
    (2, 9, 16, 4, 128, 128, False, BF16, 1 << 20, True), (1, 33, 5, 1, 128, 128, True, BF16, (1 << 30) + 77, False),
    (4, 7, 3, 3, 96, 48, False, F32, 12345, True), (2, 8, 2, 1, 256, 256, True, BF16, 3, True),
    (1, 6, 7, 2, 256, 64, False, F32, 999, True), (2, 4, 2, 2, 48, 16, True, F32, 31, True),
    (1, 4500, 2, 1, 64, 64, False, BF16, 100, True), (3, 5600, 1, 1, 32, 32, False, BF16, 0, True),
]


@pytest.mark.parametrize("B,L,H,KV,d,rot,nb,dtype,start,weights", CASES)
def test_forward_and_backward(B, L, H, KV, d, rot, nb, dtype, start, weights):
    qkv, wq, wk, inv, pos, dq, dk = make(B, L, H, KV, d, rot, dtype, L + d, start, weights)
    cqkv, cwq, cwk, cinv, cpos, cdq, cdk = cuda(qkv, wq, wk, inv, pos, dq, dk)
    q, k = cqkv[:, :, :H], cqkv[:, :, H:H + KV]
    kw = dict(inv_freq=cinv, pos=cpos, neighbours=nb)
    oq, ok = nan((B, L, H, d), dtype), nan((B, L, KV, d), dtype)
    got = ssm.qk_norm_fwd(q, k, cwq, cwk, **kw, q_out=oq, k_out=ok)
    assert got[0] is oq and got[1] is ok
    leaves = [ref.f64(t) for t in (qkv[:, :, :H], qkv[:, :, H:H + KV])]
    weights64 = [torch.ones(d, dtype=torch.float64) if w is None else ref.f64(w) for w in (wq, wk)]
    for t in leaves + weights64:
        t.requires_grad_(True)
    outs = [ref.qk_norm(x, w, inv, pos, 1e-6, nb) for x, w in zip(leaves, weights64)]
    for t, w, n in zip(got, outs, "qk"):
        w = w.detach()
        ref.close(t, w, (U * w.abs() if dtype == BF16 else 0.0) + SMALL * w.abs().amax(-1, keepdim=True), n)
    both = (outs[0] * ref.f64(dq)).sum() + (outs[1] * ref.f64(dk)).sum()
    want = torch.autograd.grad(both, leaves + weights64)
    o = {"dq": nan((B, L, H, d), dtype), "dk": nan((B, L, KV, d), dtype), "dwq": nan((d,)), "dwk": nan((d,))}
    grads = ssm.qk_norm_bwd(q, k, cwq, cwk, cdq, cdk, **kw, out=o)
    assert all(t is o[n] for t, n in zip(grads, o))
    for t, w, g, x, n in zip(grads, want, (dq, dk), leaves, ("dq", "dk")):
        # terms: rstd of the row times the gradient's largest
        size = (ref.f64(g).abs().amax(-1, keepdim=True) * 4 / (x.detach().pow(2).mean(-1, keepdim=True) + 1e-6).sqrt())
        ref.close(t, w, (U * w.abs() if t.dtype == BF16 else 0.0) + SMALL * size, n)
    for t, w, g, n in zip(grads[2:], want[2:], (dq, dk), ("dwq", "dwk")):
        # float32 sums of B L heads terms of at most 4 |dy| in a tree of runs: 2^-18 of the terms' root sum of squares
        # times 2^4 for their spread
        size = 16 * float(ref.f64(g).pow(2).sum(-1).sum().sqrt())
        ref.close(t, w, 2.0 ** -18 * size, n)
    again = ssm.qk_norm_bwd(q, k, cwq, cwk, cdq, cdk, **kw)
    assert all(torch.equal(a, b) for a, b in zip(again, grads))
    if start == 0 and rot:   # positions left out count from 0
        first = torch.arange(L, dtype=torch.int32).expand(B, L)
        plain = ssm.qk_norm_fwd(q, k, cwq, cwk, inv_freq=cinv, neighbours=nb)
        given = ssm.qk_norm_fwd(q, k, cwq, cwk, inv_freq=cinv, pos=first.contiguous().cuda(), neighbours=nb)
        assert all(torch.equal(a, b) for a, b in zip(plain, given))


def test_in_place_and_side_by_side():
    """Outputs in the inputs' place, within one fused tensor; and gradients side by side in another."""
    qkv, wq, wk, inv, pos, dq, dk = make(2, 6, 4, 2, 64, 64, BF16, 3)
    c, cwq, cwk, cinv, cpos, cdq, cdk = cuda(qkv, wq, wk, inv, pos, dq, dk)
    kw = dict(inv_freq=cinv, pos=cpos)
    want = ssm.qk_norm_fwd(c[:, :, :4], c[:, :, 4:6], cwq, cwk, **kw)
    grads = ssm.qk_norm_bwd(c[:, :, :4], c[:, :, 4:6], cwq, cwk, cdq, cdk, **kw)
    fused = nan(c.shape, BF16)
    ssm.qk_norm_bwd(c[:, :, :4], c[:, :, 4:6], cwq, cwk, cdq, cdk, **kw, out={"dq": fused[:, :, :4], "dk": fused[:, :, 4:6]})
    assert torch.equal(fused[:, :, :4], grads[0]) and torch.equal(fused[:, :, 4:6], grads[1]) and fused[:, :, 6:].isnan().all()
    values = c[:, :, 6:].clone()
    got = ssm.qk_norm_fwd(c[:, :, :4], c[:, :, 4:6], cwq, cwk, **kw, q_out=c[:, :, :4], k_out=c[:, :, 4:6])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(c[:, :, 6:], values)
    with pytest.raises(ssm.SsmError, match="overlaps"):
        ssm.qk_norm_fwd(c[:, :, :4], c[:, :, 4:6], q_out=c[:, :, 1:5])
    with pytest.raises(ssm.SsmError, match="overlaps"):
        ssm.qk_norm_fwd(c[:, :, :4], c[:, :, 4:6], k_out=c[:, :, 3:5])


def test_step_and_unit_heads():
    qkv, _, _, inv, pos, _, _ = make(5, 1, 4, 2, 128, 128, BF16, 9, 1 << 19)
    c, cinv, cpos = cuda(qkv, inv, pos)
    whole = ssm.qk_norm_fwd(c[:, :, :4], c[:, :, 4:6], inv_freq=cinv, pos=cpos)
    step = ssm.qk_norm_fwd(c[:, 0, :4], c[:, 0, 4:6], inv_freq=cinv, pos=cpos[:, 0].contiguous())
    assert torch.equal(step[0], whole[0][:, 0]) and torch.equal(step[1], whole[1][:, 0])
    unit = torch.full((128,), 128 ** -0.5, device="cuda")
    q, k = ssm.qk_norm_fwd(c[:, :, :4], c[:, :, 4:6], unit, unit)
    assert ((q.double().norm(dim=-1) - 1).abs() <= U).all() and ((k.double().norm(dim=-1) - 1).abs() <= U).all()
    zero = ssm.qk_norm_fwd(torch.zeros_like(c[:, :, :4]), torch.zeros_like(c[:, :, 4:6]))
    assert not zero[0].any() and not zero[1].any()


def test_backward_against_differences():
    qkv, wq, wk, inv, pos, dq, dk = make(1, 5, 2, 1, 32, 16, F32, 21, 50)
    grads = ssm.qk_norm_bwd(*cuda(qkv[:, :, :2], qkv[:, :, 2:3], wq, wk, dq, dk), inv_freq=inv.cuda(), pos=pos.cuda())
    at = [ref.f64(t) for t in (qkv[:, :, :2], qkv[:, :, 2:3], wq, wk)]

    def loss(q, k, wq, wk):
        return float((ref.qk_norm(q, wq, inv, pos, 1e-6, False) * dq.double()).sum()
                     + (ref.qk_norm(k, wk, inv, pos, 1e-6, False) * dk.double()).sum())

    for n, t in enumerate(grads):
        for j in torch.randint(t.numel(), (6,), generator=torch.Generator().manual_seed(n)).tolist():
            up, down = [x.clone() for x in at], [x.clone() for x in at]
            up[n].view(-1)[j] += 1e-5
            down[n].view(-1)[j] -= 1e-5
            want = (loss(*up) - loss(*down)) / 2e-5
            assert abs(float(t.view(-1)[j]) - want) <= 1e-5 * max(1.0, float(t.abs().max())), (n, j)
