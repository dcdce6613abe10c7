"""Calls of libssm_delta as programs make them: repeated, on other streams, in
captured graphs, two at once, on views of far-apart rows and long caches, on
nothing at all; and what the binding refuses."""
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


def gdr_inputs(B, L, nqk, H, K, V, seed=0, gates=F32):
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.nn.functional.normalize(torch.randn(B, L, nqk, K, generator=g), dim=-1).to(BF16) for _ in range(2))
    v = torch.randn(B, L, H, V, generator=g).to(BF16)
    dec = (-0.1 * torch.rand(B, L, H, generator=g)).to(gates)
    beta = torch.rand(B, L, H, generator=g).to(gates)
    return [t.cuda() for t in (q, k, v, dec, beta, torch.randn(B, H, V, K, generator=g), torch.randn(B, L, H, V, generator=g).to(BF16))]


def qk_inputs(B, L, H, KV, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return [t.cuda() for t in (r(B, L, H, d).to(BF16), r(B, L, KV, d).to(BF16), r(d), r(d), torch.rand(d // 2, generator=g),
                               r(B, L, H, d).to(BF16), r(B, L, KV, d).to(BF16))]


def gdr_train(seed, *sizes):
    q, k, v, g, beta, h0, dy = gdr_inputs(*(sizes or (2, 150, 2, 4, 128, 64)), seed, BF16)

    def run():
        y, last, states = ssm.gdr_fwd(q, k, v, g, beta, h0=h0, return_states=True)
        return y, last, *ssm.gdr_bwd(q, k, v, g, beta, states, dy, dh_last=last)
    return [q, k, v, g, beta, h0, dy], run


def gdr_long(seed):
    """Of few heads: cut into segments."""
    args = gdr_inputs(1, 5000, 1, 2, 64, 128, seed)[:6]
    return args, lambda: ssm.gdr_fwd(*args[:5], h0=args[5])


def gdr_train_long(seed):
    return gdr_train(seed, 1, 1500, 1, 2, 128, 64)


def gdr_step(seed):
    q, k, v, g, beta, h0, _ = gdr_inputs(5, 1, 2, 6, 128, 128, seed)
    args = [*(t[:, 0].contiguous() for t in (q, k, v, g, beta)), h0]
    return args, lambda: ssm.gdr_step(*args[:5], args[5], h_out=torch.empty_like(args[5]))


def qk_train(seed):
    q, k, wq, wk, f, dq, dk = args = qk_inputs(3, 700, 4, 2, 80, seed)
    return args, lambda: (*ssm.qk_norm_fwd(q, k, wq, wk, inv_freq=f), *ssm.qk_norm_bwd(q, k, wq, wk, dq, dk, inv_freq=f))


def swa_step(seed):
    q, k, _, _, _, _, v = qk_inputs(3, 1, 8, 2, 128, seed)
    prompt = qk_inputs(3, 900, 2, 2, 128, seed)
    cache = ssm.swa_q8_cache(3, 2, 512, 128, sinks=3)
    for t in cache:
        t.zero_()
    ssm.swa_q8_fill(prompt[0], prompt[1], cache, sinks=3)
    pos = torch.tensor([900, -1, 3 + 64 * 15 - 1], dtype=torch.int32, device="cuda")
    args = [q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(), pos, *cache]
    # (The same token again and again: the cache it leaves is the same each time.)
    return args, lambda: (ssm.swa_q8_step(*args[:3], ssm.SwaQ8Cache(*args[4:]), args[3], sinks=3), *[t.clone() for t in args[4:]])


def swa_fill(seed):
    prompt = qk_inputs(2, 333, 3, 3, 64, seed)
    lengths = torch.tensor([333, 200], dtype=torch.int32, device="cuda")

    def run():
        cache = ssm.swa_q8_cache(2, 3, 128, 64, sinks=5)
        for t in cache:
            t.zero_() if t.dtype != torch.float8_e4m3fn else t.view(torch.uint8).zero_()
        ssm.swa_q8_fill(prompt[0], prompt[1], cache, sinks=5, lengths=lengths)
        return tuple(cache)
    return [prompt[0], prompt[1]], run


def bits(outs):
    return [t.contiguous().view(torch.uint8).clone() for t in outs]


def same(a, b):
    assert len(a) == len(b)
    for n, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x, y), n


OPS = [gdr_train, gdr_train_long, gdr_long, gdr_step, qk_train, swa_step, swa_fill]


@pytest.mark.parametrize("make", OPS)
def test_repeats_bit_for_bit_and_on_another_stream(make):
    _, run = make(1)
    want = bits(run())
    same(bits(run()), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.current_stream().wait_stream(side)
    same(bits(got), want)


@pytest.mark.parametrize("make", OPS)
def test_two_captured_graphs(make):
    """Each with workspaces of its own; replayed in turn and at once, with other work between, on changed inputs."""
    calls = [make(seed) for seed in (2, 3)]
    graphs, outs = [], []
    for args, run in calls:
        run()
    torch.cuda.synchronize()
    for args, run in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run())
        graphs.append(graph)
    side = torch.cuda.Stream()
    for turn in range(3):
        for args, _ in calls:
            args[0].copy_(torch.roll(args[0], 1, -1))
        want = [bits(run()) for _, run in calls]
        torch.cuda.synchronize()
        if turn < 2:
            for graph in graphs:
                graph.replay()
        else:
            side.wait_stream(torch.cuda.current_stream())
            graphs[0].replay()
            with torch.cuda.stream(side):
                graphs[1].replay()
            torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            same(bits(got), w)


@pytest.mark.parametrize("make", OPS)
def test_two_calls_at_once(make):
    (_, one), (_, two) = make(4), make(5)
    want = [bits(one()), bits(two())]
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        a = one()
        with torch.cuda.stream(side):
            b = two()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        same(bits(a), want[0])
        same(bits(b), want[1])


def test_stream_argument():
    args, run = gdr_train(6)
    want = bits(run())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    q, k, v, g, beta, h0, dy = args
    y, last, states = ssm.gdr_fwd(q, k, v, g, beta, h0=h0, return_states=True, stream=side)
    got = ssm.gdr_bwd(q, k, v, g, beta, states, dy, dh_last=last, stream=side)
    side.synchronize()
    same(bits((y, last, *got)), want)


def far(t, token=1 << 24):
    """t's rows, (1, L, ...), `token` elements apart."""
    flat = t.flatten(2)
    room = torch.empty((t.shape[1] - 1) * token + flat.shape[2], dtype=t.dtype, device="cuda")
    view = room.as_strided(flat.shape, (0, token, 1))
    view.copy_(flat)
    return view.unflatten(-1, t.shape[2:])


def test_rows_far_apart():
    """Token strides of 2^24 elements over 200 tokens: offsets past 2^32 bytes; the same bits as on dense rows."""
    L = 200
    q, k, v, g, beta, h0, dy = gdr_inputs(1, L, 2, 2, 64, 64, 7)
    want = ssm.gdr_fwd(q, k, v, g, beta, h0=h0, return_states=True)
    fq, fk, fv = far(q), far(k), far(v)
    got = ssm.gdr_fwd(fq, fk, fv, g, beta, h0=h0, return_states=True)
    same(bits(got[:2]), bits(want[:2]))
    same(bits(ssm.gdr_bwd(fq, fk, fv, g, beta, got[2], dy)), bits(ssm.gdr_bwd(q, k, v, g, beta, want[2], dy)))
    same(bits(ssm.qk_norm_fwd(fq, fk)), bits(ssm.qk_norm_fwd(q, k)))
    want = ssm.qk_norm_fwd(q, k, eps=0.5)
    ssm.qk_norm_fwd(q, k, eps=0.5, q_out=fq, k_out=fk)
    same(bits((fq, fk)), bits(want))
    caches = []
    for keys, values in ((k, v), (far(k), fv)):
        cache = ssm.swa_q8_cache(1, 2, 64, 64)
        for t in cache:
            t.view(torch.uint8).zero_()
        ssm.swa_q8_fill(keys, values, cache)
        caches.append(bits(cache))
    same(*caches)


def test_states_past_4_gib():
    """A step over, and a forward that saves, more than 2^32 bytes: the last rows as in a call of their own."""
    B, few = 2112, 16
    q, k, v, g, beta, h0, dy = gdr_inputs(few, 3, 4, 32, 128, 128, 8)
    many = lambda t: torch.cat([t.new_zeros(B - few, *t.shape[1:]), t])
    one = lambda t: t[:, 0].contiguous()
    y, h = ssm.gdr_step(*map(one, (q, k, v, g, beta)), h0, h_out=torch.empty_like(h0))
    state = many(h0)
    assert state.numel() * 4 > 1 << 32
    got, state = ssm.gdr_step(*(many(one(t)) for t in (q, k, v, g, beta)), state)
    same(bits((got[-few:], state[-few:])), bits((y, h)))
    assert not got[:-few].any() and not state[:-few].any()
    y, h, saved = ssm.gdr_fwd(q, k, v, g, beta, h0=h0, return_states=True)
    grads = ssm.gdr_bwd(q, k, v, g, beta, saved, dy, dh_last=h)
    big = [many(t) for t in (q, k, v, g, beta)]
    got_y, got_h, got_saved = ssm.gdr_fwd(*big, h0=many(h0), return_states=True)
    assert got_saved.numel() > 1 << 32
    same(bits((got_y[-few:], got_h[-few:])), bits((y, h)))
    got = ssm.gdr_bwd(*big, got_saved, many(dy), dh_last=many(h))
    same(bits([t[-few:] for t in got]), bits(grads))


def test_a_cache_past_4_gib():
    """The last row's part of the rings lies behind 2^32 bytes; the other rows have no token."""
    B, KV, H, d, window, sinks = 18, 8, 16, 128, 1 << 18, 2
    cache = ssm.swa_q8_cache(B, KV, window, d, sinks=sinks)
    assert cache.k_ring.numel() > 1 << 32
    g, on = torch.Generator().manual_seed(9), torch.Generator("cuda").manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g).to(BF16).cuda()
    pos = torch.full((B,), -1, dtype=torch.int32)
    pos[-1] = at = sinks + 64 * (window // 64 * 3 + 5) + 20
    for t in cache[2:]:
        t.view(torch.uint8)[:-1] = 0x7f       # NaN
    for ring, scale, near in zip(cache[2:4], cache[4:6], cache[:2]):
        for c in range(KV):
            ring[-1, c] = (torch.randn(window, d, device="cuda", generator=on) * 50).to(torch.float8_e4m3fn)
        scale[-1] = torch.rand(KV, window // 64, generator=g).cuda() / 50
        near[-1] = r(KV, sinks + 64, d)
    q, k, v = r(B, H, d), r(B, KV, d), r(B, KV, d)
    before = [t[:-1].clone() for t in cache[:2]]
    y = ssm.swa_q8_step(q, k, v, cache, pos.cuda(), sinks=sinks)
    assert not y[:-1].any()
    for t, was in zip(cache[:2], before):
        assert torch.equal(t[:-1].view(torch.uint8), was.view(torch.uint8))
    block = (at - sinks) // 64 % (window // 64)
    seen = torch.ones(window, dtype=torch.bool, device="cuda")
    seen[64 * block:64 * block + 21] = False
    for h in range(H):
        c = h * KV // H
        keys, values = (torch.cat([ring[-1, c][seen].float() * scale[-1, c].repeat_interleave(64)[seen, None],
                                   near[-1, c, :sinks + 21].float()]) for ring, scale, near in zip(cache[2:4], cache[4:6], cache[:2]))
        p = torch.softmax((keys.double() @ q[-1, h].double()) * d ** -0.5, 0)
        want, size = p @ values.double(), p @ values.double().abs()
        # Scores of size 2^6 at most, held to 2^-19 of that; weights in two parts, 2^-16; y's own rounding.
        ref.close(y[-1, h], want.cpu(), (U * want.abs() + (2.0 ** -14 + 2.0 ** -13) * size).cpu(), h)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
def test_any_scale(scale):
    """y is linear in it; so are the gradients that pass through y."""
    q, k, v, g, beta, h0, dy = gdr_inputs(1, 100, 1, 2, 64, 64, 10)
    args = [ref.f64(t) for t in (q, k, v, g, beta)]
    y, last, states = ssm.gdr_fwd(q, k, v, g, beta, h0=h0, scale=scale, return_states=True)
    want, want_last, _, size = ref.gdr(*args, ref.f64(h0), None, scale)
    # As for the usual scale: values of about 1 besides the state's, times |q| = 1 and the scale.
    ref.close(y, want, U * want.abs() + 2.0 ** -13 * (size + abs(scale)), "y")
    got = ssm.gdr_bwd(q, k, v, g, beta, states, dy, scale=scale)
    grads, sizes = ref.gdr_bwd(*args, ref.f64(dy), ref.f64(h0), None, scale)
    for t, name in zip(got, ("dq", "dk", "dv", "dg", "dbeta")):
        bound = U * grads[name].abs() if t.dtype == BF16 else 0
        size = sizes[name] if grads[name].dim() == 3 else sizes[name].unflatten(2, (grads[name].shape[2], -1)).sum(3)[..., None]
        ref.close(t, grads[name], bound + 2.0 ** -14 * size, name)
    y, _ = ssm.gdr_step(*(t[:, 0].contiguous() for t in (q, k, v, g, beta)), h0, scale=scale, h_out=torch.empty_like(h0))
    want, _, _, size = ref.gdr(*(t[:, :1] for t in args), ref.f64(h0), None, scale)
    ref.close(y, want[:, 0], U * want[:, 0].abs() + 2.0 ** -19 * (size[:, 0] + 4 * abs(scale)), "step")


def test_nothing():
    """No tokens, no rows: states pass through, and gradients of weights are zero."""
    q, k, v, g, beta, h0, dy = gdr_inputs(2, 1, 1, 2, 64, 128, 11)
    none = [t[:, :0] for t in (q, k, v, g, beta, dy)]
    y, last, states = ssm.gdr_fwd(*none[:5], h0=h0, return_states=True)
    assert y.shape == (2, 0, 2, 128) and torch.equal(last, h0) and states.numel() == 0
    assert not ssm.gdr_fwd(*none[:5])[1].any()
    assert torch.equal(ssm.gdr_bwd(*none[:5], states, none[5], dh_last=h0)[5], h0)
    rows = [t[:0] for t in (q, k, v, g, beta, h0)]
    assert ssm.gdr_fwd(*rows[:5], h0=rows[5])[1].shape == (0, 2, 128, 64)
    assert ssm.gdr_step(*(t[:, 0] for t in rows[:5]), rows[5])[0].shape == (0, 2, 128)
    q, k, wq, wk, f, dq, dk = qk_inputs(2, 1, 4, 2, 64, 11)
    junk = {n: torch.full((64,), float("nan"), device="cuda") for n in ("dwq", "dwk")}
    outs = ssm.qk_norm_bwd(q[:, :0], k[:, :0], wq, wk, dq[:, :0], dk[:, :0], inv_freq=f, out=junk)
    assert outs[0].shape == (2, 0, 4, 64) and not outs[2].any() and not outs[3].any()
    assert ssm.qk_norm_fwd(q[:0], k[:0], inv_freq=f)[1].shape == (0, 1, 2, 64)
    cache = ssm.swa_q8_cache(0, 2, 64, 64)
    assert ssm.swa_q8_step(q[:0, 0], k[:0, 0], k[:0, 0], cache, torch.empty(0, dtype=torch.int32, device="cuda")).shape == (0, 4, 64)
    cache = ssm.swa_q8_cache(2, 2, 64, 64)
    for t in cache:
        t.view(torch.uint8).fill_(3)
    ssm.swa_q8_fill(k[:, :0], k[:, :0], cache)
    ssm.swa_q8_fill(k, k, cache, lengths=torch.tensor([0, -5], dtype=torch.int32, device="cuda"))
    assert all((t.view(torch.uint8) == 3).all() for t in cache)


def test_last_state_in_place_of_the_first():
    for L in (70, 5000):
        q, k, v, g, beta, h0, _ = gdr_inputs(1, L, 1, 2, 64, 64, 12)
        want = ssm.gdr_fwd(q, k, v, g, beta, h0=h0)
        h = h0.clone()
        got = ssm.gdr_fwd(q, k, v, g, beta, h0=h, h_last=h)
        assert got[1] is h
        same(bits(got), bits(want))


def test_dims_of_mismatched_tensors():
    """What the binding makes of shapes, types and strides, and refuses."""
    from state_space_model_ssm_amd import delta
    z = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype, device="cuda")
    b = lambda *s: z(*s, dtype=BF16)
    q, v, g = b(2, 5, 2, 64), b(2, 5, 4, 64), z(2, 5, 4)
    d = delta._gdr_dims(q, q, v, g, g, None, 2)
    assert (d.batch, d.seqlen, d.nqk, d.nheads, d.kdim, d.vdim, d.q_token, d.v_batch, d.scale, d.gate_dtype) == (2, 5, 2, 4, 64, 64, 128, 1280, 0.125, 0)
    for bad in ((q.float(), q, v, g, g), (q, q, v.float(), g, g), (q, q, v, g.half(), g.half())):
        with pytest.raises(TypeError):
            delta._gdr_dims(*bad, None, 2)
    for bad in ((q, q[:, :4], v, g, g), (q, q, v[:1], g, g), (q, q, v, g[:, :4], g), (q[0], q[0], v, g, g), (q, q, v, g, g.bfloat16())):
        with pytest.raises(ValueError):
            delta._gdr_dims(*bad, None, 2)
    with pytest.raises(ValueError):   # heads that are not adjacent
        delta._gdr_dims(b(2, 2, 5, 64).transpose(1, 2), q, v, g, g, None, 2)
    n = lambda q, k, wq=None, wk=None, f=None, pos=None: delta._qk_norm_dims(q, k, wq, wk, f, pos, 1e-6, False, q, k, True, True)
    assert n(q, v, f=z(32)).rot == 64 and n(q, v).rot == 0
    with pytest.raises(TypeError, match="k must have"):
        n(q, v.float())
    with pytest.raises(TypeError):
        n(q.half(), v.half())
    with pytest.raises(ValueError, match="one device"):
        ssm.gdr_fwd(q, q, v, g, g.cpu())
    with pytest.raises(ValueError, match="one device"):
        ssm.gdr_step(q[:, 0], q[:, 0], v[:, 0], g[:, 0].contiguous(), g[:, 0].contiguous(), torch.zeros(2, 4, 64, 64))
    with pytest.raises(ValueError, match="contiguous"):
        ssm.gdr_fwd(q, q, v, g, z(2, 4, 5).mT)
    with pytest.raises(ssm.SsmError, match="multiples of 8"):
        ssm.gdr_fwd(b(2, 5, 132)[..., :128].unflatten(-1, (2, 64)), q, v, g, g)
    with pytest.raises(ssm.SsmError, match="aligned"):
        ssm.qk_norm_fwd(b(2 * 5 * 128 + 1)[1:].view(2, 5, 2, 64), v)
    for bad in (dict(q=q, k=v[:, :4]), dict(q=q, k=b(2, 5, 4, 32)), dict(q=q, k=v, wq=z(32)), dict(q=q, k=v, f=z(4, 8)),
                dict(q=q, k=v, f=z(32), pos=z(2, 4, dtype=torch.int32)), dict(q=q[0, 0], k=v[0, 0])):
        with pytest.raises(ValueError):
            n(**bad)
    with pytest.raises(ValueError, match="pos is required"):
        n(q[:, 0], v[:, 0], f=z(32))
    cache = ssm.swa_q8_cache(2, 2, 128, 64, sinks=3)
    assert delta._q8_cache(cache, 2, 2, 64, 3) == 128
    for kw in ((2, 2, 64, 4), (1, 2, 64, 3), (2, 4, 64, 3), (2, 2, 128, 3)):
        with pytest.raises(ValueError):
            delta._q8_cache(cache, *kw)
    with pytest.raises(ValueError):
        delta._q8_cache(cache._replace(v_ring=cache.v_ring.view(torch.uint8)), 2, 2, 64, 3)
    with pytest.raises(ValueError, match="multiple of 64"):
        delta._q8_cache(cache._replace(k_ring=cache.k_ring[:, :, :100]), 2, 2, 64, 3)
