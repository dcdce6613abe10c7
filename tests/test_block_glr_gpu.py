"""The gated linear recurrence (forward, backward, step) against float64."""
import numpy as np
import pytest
import torch

import block_reference as ref
import state_space_model_ssm_amd as ssm

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(batch, L, dim, dtype, seed, resets=False, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x, rec, inp, dy = ((torch.randn(batch, L, dim, generator=g) * scale).to(dtype) for _ in range(4))
    A = -torch.exp(torch.rand(dim, generator=g) * 7.0 - 5.5)
    h0, dh = torch.randn(batch, dim, generator=g), torch.randn(batch, dim, generator=g)
    reset = (torch.rand(batch, L, generator=g) < 0.1).to(torch.uint8) if resets else None
    return x, rec, inp, A, dy, h0, dh, reset


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def nan(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


CASES = [  # batch, L, dim, dtype, out dtype, resets, h0
    (1, 1, 1, F32, F32, False, True), (2, 1, 5, BF16, BF16, True, True), (1, 2, 64, BF16, F32, False, False),
    (3, 15, 63, F32, F32, True, True), (1, 16, 65, BF16, BF16, False, True), (2, 17, 130, BF16, BF16, True, False),
    (1, 31, 2, F32, BF16, False, True), (1, 63, 66, BF16, BF16, True, True), (2, 64, 96, F32, F32, False, True),
    (1, 127, 257, F32, F32, True, True), (1, 129, 256, BF16, BF16, True, True), (2, 300, 31, BF16, BF16, False, True),
    (1, 1000, 72, F32, F32, True, True), (1, 2500, 34, BF16, BF16, True, True), (1, 4097, 8, F32, F32, False, True),
    (3, 513, 512, BF16, BF16, True, True), (1, 8192, 64, BF16, BF16, True, True), (130, 33, 33, BF16, BF16, True, True),
]


@pytest.mark.parametrize("batch,L,dim,dtype,out,resets,with_h0", CASES)
def test_forward_and_backward(batch, L, dim, dtype, out, resets, with_h0):
    x, rec, inp, A, dy, h0, dh, reset = make(batch, L, dim, dtype, L * 1000 + dim, resets)
    h0 = h0 if with_h0 else None
    cx, crec, cinp, cA, cdy, ch0, cdh, creset = cuda(x, rec, inp, A, dy, h0, dh, reset)
    y, hl, st = nan((batch, L, dim), out), nan((batch, dim), F32), nan((batch, -(-L // 16), dim), F32)
    got = ssm.glr_fwd(cx, crec, cinp, cA, h0=ch0, reset=creset, out_dtype=out, return_states=True, y=y, h_last=hl,
                      states=st)
    assert got[0] is y and got[1] is hl and got[2] is st
    h, last, _ = ref.glr(x, rec, inp, A, h0, reset)
    ref.assert_close(y, h, ref.storage_tol(h, out), "y")
    ref.assert_close(hl, last, ref.storage_tol(h, F32), "h_last")
    start = np.zeros((batch, 1, dim)) if h0 is None else ref.f64(h0)[:, None]
    ref.assert_close(st, np.concatenate([start, h[:, :-1]], 1)[:, ::16], ref.storage_tol(h, F32), "states")

    outs = {k: nan((batch, L, dim), dtype) for k in ("dx", "drec", "dinp")}
    outs |= {"dA": nan((dim,), F32), "dh0": nan((batch, dim), F32)}
    got = ssm.glr_bwd(cx, crec, cinp, cA, st, cdy, dh_last=cdh, reset=creset, out=outs)
    want, size = ref.glr_bwd(x, rec, inp, A, dy, h0, reset, dh)
    for k, t in zip(("dx", "drec", "dinp", "dA", "dh0"), got):
        ref.assert_close(t, want[k], ref.storage_tol(want[k], t.dtype, size.get(k)), k)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gates_at_their_ends(dtype):
    """Gates driven to 0 and 1, decays down to 0, and a gate that shuts: no NaN, no lost digits."""
    x, rec, inp, A, dy, h0, dh, _ = make(2, 70, 40, dtype, 5)
    rec = torch.linspace(-120, 120, 70)[None, :, None].expand(2, 70, 40).to(dtype).contiguous()
    inp = torch.linspace(110, -110, 70)[None, :, None].expand(2, 70, 40).to(dtype).contiguous()
    A = -torch.logspace(-7, 3, 40)
    args = cuda(x, rec, inp, A)
    y, hl, st = ssm.glr_fwd(*args, h0=h0.cuda(), return_states=True)
    h, last, _ = ref.glr(x, rec, inp, A, h0)
    ref.assert_close(y, h, ref.storage_tol(h, dtype), "y")
    got = ssm.glr_bwd(*args, st, dy.cuda(), dh_last=dh.cuda())
    want, size = ref.glr_bwd(x, rec, inp, A, dy, h0, None, dh)
    for k, t in zip(("dx", "drec", "dinp", "dA", "dh0"), got):
        ref.assert_close(t, want[k], ref.storage_tol(want[k], t.dtype, size.get(k)), k)


def test_small_decay_rates_keep_their_digits():
    """1 - a^2 where a rounds close to 1: relative error of y, channel by channel."""
    x, rec, inp, _, _, _, _, _ = make(1, 48, 24, F32, 9)
    A = -torch.logspace(-9, -1, 24)
    y, _ = ssm.glr_fwd(*cuda(x, rec, inp, A))
    h, _, _ = ref.glr(x, rec, inp, A)
    ref.assert_close(y, h, 1e-5 * np.abs(h).max(axis=(0, 1), keepdims=True), "y")


def test_backward_against_differences():
    x, rec, inp, A, dy, h0, dh, reset = (None if t is None else t.double() for t in make(1, 20, 3, F32, 3, True))
    h32 = [t.float().cuda() for t in (x, rec, inp, A)]
    st = ssm.glr_fwd(*h32, h0=h0.float().cuda(), reset=reset.to(torch.uint8).cuda(), return_states=True)[2]
    got = ssm.glr_bwd(*h32, st, dy.float().cuda(), dh_last=dh.float().cuda(), reset=reset.to(torch.uint8).cuda())

    def loss(x, rec, inp, A, h0):
        h, last, _ = ref.glr(x, rec, inp, A, h0, reset)
        return float((h * dy.numpy()).sum() + (last * dh.numpy()).sum())

    at, eps = [x, rec, inp, A, h0], 1e-5
    for k, t in enumerate(got):
        for j in np.random.default_rng(k).integers(0, t.numel(), 6):
            up, down = [v.clone() for v in at], [v.clone() for v in at]
            up[k].view(-1)[j] += eps
            down[k].view(-1)[j] -= eps
            # Central differences: eps^2 of third derivatives of order 1, and 1e-16 / eps of the loss.
            want = (loss(*up) - loss(*down)) / (2 * eps)
            assert abs(float(t.view(-1)[j]) - want) <= 1e-5 * max(1.0, float(t.abs().max())), (k, j)


@pytest.mark.parametrize("batch,dim,dtype,out", [(1, 1, F32, F32), (3, 65, BF16, BF16), (64, 320, BF16, F32),
                                                 (2, 100, F32, BF16)])
def test_step(batch, dim, dtype, out):
    x, rec, inp, A, _, h0, _, _ = make(batch, 1, dim, dtype, 11)
    h, last, _ = ref.glr(x, rec, inp, A, h0)
    c = cuda(x[:, 0].contiguous(), rec[:, 0].contiguous(), inp[:, 0].contiguous(), A)
    state = h0.cuda()
    new = nan((batch, dim), F32)
    y, hn = ssm.glr_step(*c, state, h_out=new, out_dtype=out)
    assert hn is new and torch.equal(state.cpu(), h0)
    ref.assert_close(y, last, ref.storage_tol(last, out), "y")
    ref.assert_close(new, last, ref.storage_tol(last, F32), "h_out")
    y2, same = ssm.glr_step(*c, state, out_dtype=out)
    assert same is state and torch.equal(state, new) and torch.equal(y, y2)


def test_a_sequence_in_pieces_and_steps():
    x, rec, inp, A, _, h0, _, _ = make(2, 90, 70, F32, 13)
    c = cuda(x, rec, inp, A)
    y, hl = ssm.glr_fwd(*c, h0=h0.cuda())
    state = h0.cuda()
    parts = []
    for lo, hi in ((0, 37), (37, 88)):
        piece, state = ssm.glr_fwd(*(t[:, lo:hi].contiguous() for t in c[:3]), c[3], h0=state, h_last=state)
        parts.append(piece)
    for t in (88, 89):
        piece, state = ssm.glr_step(*(v[:, t].contiguous() for v in c[:3]), c[3], state)
        parts.append(piece[:, None])
    ref.assert_close(torch.cat(parts, 1), ref.f64(y), 2e-5 * float(y.abs().max()), "y")
    ref.assert_close(state, ref.f64(hl), 2e-5 * float(hl.abs().max()), "h_last")


def test_empty_sequences():
    A = -torch.ones(8, device="cuda")
    z = torch.empty(2, 0, 8, device="cuda")
    h0 = torch.randn(2, 8, device="cuda")
    y, hl, st = ssm.glr_fwd(z, z, z, A, h0=h0, return_states=True)
    assert y.shape == (2, 0, 8) and st.shape == (2, 0, 8) and torch.equal(hl, h0)
    assert torch.equal(ssm.glr_fwd(z, z, z, A)[1], torch.zeros_like(h0))
    dx, _, _, dA, dh0 = ssm.glr_bwd(z, z, z, A, st, z, dh_last=h0)
    assert dx.shape == (2, 0, 8) and not dA.any() and torch.equal(dh0, h0)
    e = torch.empty(0, 5, 8, device="cuda")
    dA = nan((8,), F32)
    ssm.glr_bwd(e, e, e, A, torch.empty(0, 1, 8, device="cuda"), e, out={"dA": dA})
    assert not dA.any()
    n = torch.empty(2, 5, 0, device="cuda")
    assert ssm.glr_fwd(n, n, n, A[:0])[0].shape == (2, 5, 0)


def test_nan_stays_in_its_channel_and_resets_stop_it():
    x, rec, inp, A, _, _, _, _ = make(1, 200, 70, F32, 17)
    x[0, 50, 3] = float("nan")
    reset = torch.zeros(1, 200, dtype=torch.bool)
    reset[0, 120] = True
    y, _ = ssm.glr_fwd(*cuda(x, rec, inp, A), reset=reset.cuda())
    bad = torch.isnan(y[0]).cpu()
    assert bad[50:120, 3].all() and int(bad.sum()) == 70
    rec[0, 60, 5] = float("nan")
    y, _ = ssm.glr_fwd(*cuda(x, rec, inp, A), reset=reset.cuda())
    assert torch.isnan(y[0, 60:120, 5]).all() and not torch.isnan(y[0, 120:]).any()


def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph():
    x, rec, inp, A, dy, h0, _, reset = make(2, 700, 200, BF16, 21, True)
    c = cuda(x, rec, inp, A, dy, h0, reset)

    def both(stream=None):
        y, hl, st = ssm.glr_fwd(*c[:4], h0=c[5], reset=c[6], return_states=True, stream=stream)
        return (y, hl, st) + ssm.glr_bwd(*c[:4], st, c[4], reset=c[6], stream=stream)

    first = [t.clone() for t in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = both(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for _ in range(3):
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, held))
        assert all(torch.equal(a, b) for a, b in zip(first, both()))


def test_offsets_past_32_bits():
    """A sequence whose tensors pass 2^31 elements: its last rows against a short run from the state before them."""
    batch, L, dim = 1, 262144 + 40, 8200
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, L, dim, generator=g, device="cuda", dtype=BF16)
    A = -torch.rand(dim, device="cuda") - 0.1
    y, hl, st = ssm.glr_fwd(x, x, x, A, return_states=True)
    tail = x[:, 262144:].contiguous()
    y2, hl2 = ssm.glr_fwd(tail, tail, tail, A, h0=st[:, 262144 // 16].contiguous())
    ref.assert_close(y[:, 262144:], ref.f64(y2), ref.storage_tol(ref.f64(y2), BF16), "y")
    ref.assert_close(hl, ref.f64(hl2), 1e-5 * float(hl2.abs().max()), "h_last")
    dx, drec, dinp, _, _ = ssm.glr_bwd(x, x, x, A, st, x)
    dx2, drec2, dinp2, _, _ = ssm.glr_bwd(tail, tail, tail, A, st[:, 262144 // 16:].contiguous(), tail)
    for a, b in ((dx, dx2), (drec, drec2), (dinp, dinp2)):
        ref.assert_close(a[:, 262144:], ref.f64(b), 2 * ref.storage_tol(ref.f64(b), BF16), "gradient")


@pytest.mark.parametrize("batch,L", [(2 ** 24 + 5, 1), (2 ** 23 + 3, 129)])
def test_tiles_past_2_24(batch, L):
    """More tiles than a launch has workgroups along one axis, of one tile per row and of two."""
    g = torch.Generator(device="cuda").manual_seed(L)
    x, rec, dy = (torch.randn(batch, L, 1, generator=g, device="cuda") for _ in range(3))
    A = torch.tensor([-0.3], device="cuda")
    h0 = torch.randn(batch, 1, generator=g, device="cuda")
    y, hl, st = ssm.glr_fwd(x, rec, x, A, h0=h0, return_states=True, y=nan(x.shape, F32), h_last=nan(h0.shape, F32))
    out = {k: nan(x.shape, F32) for k in ("dx", "drec", "dinp")} | {"dh0": nan(h0.shape, F32)}
    ssm.glr_bwd(x, rec, x, A, st, dy, out=out)

    def gates(t):
        r, i = torch.sigmoid(rec[:, t].double()), torch.sigmoid(x[:, t].double())
        a = torch.exp(A.double() * r)
        return a, torch.sqrt(-torch.expm1(2 * A.double() * r)), i

    def close(got, want):
        return bool(((got.double() - want).abs() <= 1e-5 * want.abs().max()).all())

    h = h0.double()
    for t in range(L):
        a, b, i = gates(t)
        h = a * h + b * i * x[:, t].double()
        assert close(y[:, t], h), t
    assert close(hl, h)
    carry = torch.zeros_like(h)
    for t in range(L - 1, -1, -1):
        a, b, i = gates(t)
        before = h0.double() if t == 0 else y[:, t - 1].double()
        v, d = x[:, t].double(), dy[:, t].double() + carry
        carry = a * d
        w = d * (a * before - a * a / b * i * v)
        r = torch.log(a) / A.double()
        assert close(out["dx"][:, t], d * b * i) and close(out["dinp"][:, t], d * b * v * i * (1 - i)), t
        assert close(out["drec"][:, t], w * A.double() * r * (1 - r)), t
    assert close(out["dh0"], carry)


def test_steps_and_empty_sequences_past_2_32_values():
    batch, dim = 2 ** 22 + 1, 1024
    x = torch.empty(batch, dim, device="cuda", dtype=BF16).normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    h = torch.ones(batch, dim, device="cuda")
    A = -torch.rand(dim, device="cuda")
    y, new = ssm.glr_step(x, x, x, A, h)
    for rows in (slice(0, 64), slice(batch - 64, batch)):
        part = x[rows].contiguous()
        want, state = ssm.glr_step(part, part, part, A, torch.ones(64, dim, device="cuda"))
        assert torch.equal(y[rows], want) and torch.equal(new[rows], state)
    del x, y
    empty = torch.empty(batch, 0, dim, device="cuda")
    _, last = ssm.glr_fwd(empty, empty, empty, A, h0=h, h_last=nan((batch, dim), F32))
    assert torch.equal(last[-64:], h[-64:]) and torch.equal(last[:64], h[:64])


@pytest.mark.parametrize("batch,L,dim,dtype", [(2, 300, 70, F32), (3, 300, 64, BF16), (1, 4097, 200, BF16), (2, 4097, 33, F32),
                                               (4, 2500, 2100, BF16)])
def test_state_in_place_over_several_tiles(batch, L, dim, dtype):
    """h_last given as h0 itself: every tile of the first group reads h0, the last tile overwrites it."""
    x, rec, inp, A, _, h0, _, reset = make(batch, L, dim, dtype, L + dim, True)
    c = cuda(x, rec, inp, A)
    for cut in (None, reset.cuda()):
        want, last, states = ssm.glr_fwd(*c, h0=h0.cuda(), reset=cut, return_states=True)
        state = h0.cuda()
        got, same, st = ssm.glr_fwd(*c, h0=state, h_last=state, reset=cut, return_states=True)
        assert same is state and torch.equal(state, last) and torch.equal(got, want) and torch.equal(st, states)


@pytest.mark.parametrize("batch,L,dim,dtype", [(1, 2300, 67 * 32, F32), (3, 2100, 25 * 64, BF16), (2, 4200, 33 * 32 - 5, BF16)])
def test_many_channel_blocks_over_several_groups_of_tiles(batch, L, dim, dtype):
    """64 channel blocks and more, numbers of them that no 32 counters share evenly, two groups of tiles and more, resets."""
    x, rec, inp, A, dy, h0, dh, _ = make(batch, L, dim, dtype, dim)
    reset = (torch.rand(batch, L, generator=torch.Generator().manual_seed(L)) < 1 / 200).to(torch.uint8)
    c = cuda(x, rec, inp, A, dy, h0, dh, reset)
    y, hl, st = ssm.glr_fwd(*c[:4], h0=c[5], reset=c[7], return_states=True, y=nan(x.shape, dtype))
    h, last, _ = ref.glr(x, rec, inp, A, h0, reset)
    ref.assert_close(y, h, ref.storage_tol(h, dtype), "y")
    ref.assert_close(hl, last, ref.storage_tol(h, F32), "h_last")
    got = ssm.glr_bwd(*c[:4], st, c[4], dh_last=c[6], reset=c[7], out={"dx": nan(x.shape, dtype)})
    want, size = ref.glr_bwd(x, rec, inp, A, dy, h0, reset, dh)
    for k, t in zip(("dx", "drec", "dinp", "dA", "dh0"), got):
        ref.assert_close(t, want[k], ref.storage_tol(want[k], t.dtype, size.get(k)), k)
