"""Sliding-window attention with sinks (forward, backward, step, fill) against float64."""
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


def make(B, L, H, KV, d, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    q, k, v, dy = ((torch.randn(B, L, n, d, generator=g) * s).to(BF16)
                   for n, s in ((H, std), (KV, std), (KV, 1.0), (H, 1.0)))
    return q, k, v, dy


def nan(shape, dtype=BF16):
    return torch.full(tuple(shape), float("nan"), dtype=dtype, device="cuda")


def check(q, k, v, dy, window, sinks, lengths=None, scale=None):
    c = [t.cuda() for t in (q, k, v)]
    kw = dict(window=window, sinks=sinks, scale=scale, lengths=None if lengths is None else lengths.cuda())
    B, L, H, _ = q.shape
    y, lse = nan(q.shape), nan((B, H, L), F32)
    ssm.swa_fwd(*c, **kw, y=y, lse=lse)
    want, tol = ref.swa(q, k, v, window, sinks, lengths, scale, dy)
    ref.assert_close(y, want["y"], tol["y"], "y")
    seen = np.isfinite(want["lse"])
    got = lse.cpu().double().numpy()
    assert np.array_equal(got == -np.inf, ~seen)
    assert np.all(np.abs(got[seen] - want["lse"][seen]) <= 2e-5 * np.maximum(1, np.abs(want["lse"][seen])))
    out = {n: nan(t.shape) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    ssm.swa_bwd(*c, y, lse, dy.cuda(), **kw, out=out)
    for n, t in out.items():
        ref.assert_close(t, want[n], tol[n], n)


CASES = [  # B, L, H, KV, d, window, sinks
    (1, 1, 1, 1, 64, 1, 0), (2, 3, 2, 1, 128, 2, 1), (1, 31, 4, 4, 64, 8, 0), (1, 33, 3, 1, 64, 33, 2),
    (1, 64, 8, 2, 128, 16, 4), (2, 65, 4, 2, 64, 64, 1), (1, 127, 2, 2, 128, 500, 0), (1, 128, 5, 5, 64, 1, 3),
    (1, 130, 6, 2, 128, 1, 0), (1, 200, 4, 1, 64, 63, 64), (1, 257, 8, 1, 128, 65, 70), (1, 300, 2, 1, 64, 100, 150),
    (1, 500, 16, 2, 64, 129, 4), (3, 190, 7, 7, 128, 96, 16), (1, 700, 4, 2, 128, 256, 4), (1, 1500, 2, 1, 64, 200, 1),
    (1, 1300, 4, 2, 128, 90, 140), (2, 1100, 3, 1, 64, 40, 4),
]


@pytest.mark.parametrize("B,L,H,KV,d,window,sinks", CASES)
def test_forward_and_backward(B, L, H, KV, d, window, sinks):
    check(*make(B, L, H, KV, d, L * 100 + window), window, sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sinks", [0, 3, 80])
def test_lengths(d, sinks):
    """Rows of every length, none among them; what lies past a length is not read."""
    q, k, v, dy = make(7, 150, 4, 2, d, 5)
    lengths = torch.tensor([0, 1, 63, 64, 129, 150, 400], dtype=torch.int32)
    for b, n in enumerate(lengths.tolist()):
        for t in (q, k, v):
            t[b, n:] = float("nan")
    check(q, k, v, dy, 50, sinks, lengths)
    lengths[1] = -5
    kw = dict(window=50, sinks=sinks, lengths=lengths.cuda())
    y, lse = ssm.swa_fwd(q.cuda(), k.cuda(), v.cuda(), **kw)
    assert not y[:2].any() and torch.isinf(lse[:2]).all()


@pytest.mark.parametrize("B,L,H,KV,d,window,sinks", [
    (8, 260, 4, 1, 64, 64, 3), (4, 200, 4, 2, 128, 150, 5), (2, 330, 12, 4, 64, 330, 0), (3, 520, 6, 2, 64, 100, 40),
    (1, 900, 4, 1, 64, 500, 5), (1, 900, 8, 1, 128, 500, 130), (5, 300, 2, 1, 128, 40, 2), (16, 70, 1, 1, 64, 70, 1)])
def test_rows_of_unequal_length_in_every_work_order(B, L, H, KV, d, window, sinks):
    """Key heads by rows that share out over 8 or do not, windows of less and of more than half the sequence."""
    g = torch.Generator().manual_seed(B * L)
    check(*make(B, L, H, KV, d, L + H), window, sinks, torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32))


def test_garbage_gradients_past_a_length_are_not_read():
    q, k, v, dy = make(2, 100, 2, 1, 64, 6)
    lengths = torch.tensor([40, 100], dtype=torch.int32)
    kw = dict(window=30, sinks=2, lengths=lengths.cuda())
    c = [t.cuda() for t in (q, k, v)]
    y, lse = ssm.swa_fwd(*c, **kw)
    clean = ssm.swa_bwd(*c, y, lse, dy.cuda(), **kw)
    y, lse, bad = y.clone(), lse.clone(), dy.cuda()
    y[0, 40:], lse[0, :, 40:], bad[0, 40:] = float("nan"), float("nan"), float("inf")
    assert all(torch.equal(a, b) for a, b in zip(clean, ssm.swa_bwd(*c, y, lse, bad, **kw)))


@pytest.mark.parametrize("std,scale", [(6.0, None), (0.01, None), (1.0, 0.0), (1.0, -0.3), (3.0, 1.0)])
def test_scores_of_all_sizes(std, scale):
    check(*make(1, 180, 4, 2, 64, 7, std=std if scale is None else 1.0), 70, 4, scale=scale)


def test_values_that_a_query_does_not_see_do_not_reach_it():
    """NaN and infinities in keys and values outside a query's window leave its output as it was."""
    for d in (64, 128):
        q, k, v, _ = make(1, 400, 2, 1, d, 8)
        clean, _ = ssm.swa_fwd(q.cuda(), k.cuda(), v.cuda(), window=60, sinks=2)
        k[0, 100], v[0, 100] = float("nan"), float("inf")
        v[0, 250, 0, 3] = float("-inf")
        y, _ = ssm.swa_fwd(q.cuda(), k.cuda(), v.cuda(), window=60, sinks=2)
        untouched = [t for t in range(400) if not (100 <= t < 160 or 250 <= t < 310)]
        assert torch.equal(y[:, untouched], clean[:, untouched])
        assert torch.isnan(y[0, 100:160].float()).all() and torch.isinf(y[0, 250:310, :, 3].float()).all()


def test_strided_views_of_a_fused_projection():
    B, L, H, KV, d = 2, 140, 4, 2, 64
    g = torch.Generator().manual_seed(3)
    fused = torch.randn(B, L + 3, (H + 2 * KV) * d + 8, generator=g).to(BF16).cuda()[:, 2:L + 2]
    q = fused[..., :H * d].unflatten(-1, (H, d))
    k = fused[..., H * d:(H + KV) * d].unflatten(-1, (KV, d))
    v = fused[..., (H + KV) * d:(H + 2 * KV) * d].unflatten(-1, (KV, d))
    dy = torch.randn(B, L, H, d, generator=g).to(BF16).cuda()
    kw = dict(window=33, sinks=4)
    y, lse = ssm.swa_fwd(q, k, v, **kw)
    dense = [t.contiguous() for t in (q, k, v)]
    y2, lse2 = ssm.swa_fwd(*dense, **kw)
    assert torch.equal(y, y2) and torch.equal(lse, lse2)
    assert all(torch.equal(a, b) for a, b in zip(ssm.swa_bwd(q, k, v, y, lse, dy, **kw),
                                                 ssm.swa_bwd(*dense, y, lse, dy, **kw)))
    cut = q.transpose(0, 1).contiguous().transpose(0, 1)     # token-major storage
    assert torch.equal(ssm.swa_fwd(cut, k, v, **kw)[0], y)


def test_backward_against_differences():
    q, k, v, dy = make(1, 40, 2, 1, 64, 4)
    c = [t.cuda() for t in (q, k, v)]
    y, lse = ssm.swa_fwd(*c, window=13, sinks=2)
    got = ssm.swa_bwd(*c, y, lse, dy.cuda(), window=13, sinks=2)
    tol = ref.swa(q, k, v, 13, 2, dy=dy)[1]

    def loss(q, k, v):
        return float((ref.swa(q, k, v, 13, 2)[0]["y"] * ref.f64(dy)).sum())

    for n, name in enumerate(("dq", "dk", "dv")):
        for j in np.random.default_rng(n).integers(0, got[n].numel(), 6):
            at = [[t.double().clone() for t in (q, k, v)] for _ in range(2)]
            at[0][n].view(-1)[j] += 1e-4
            at[1][n].view(-1)[j] -= 1e-4
            want = (loss(*at[0]) - loss(*at[1])) / 2e-4
            assert abs(float(got[n].view(-1)[j]) - want) <= tol[name].reshape(-1)[j] + 1e-5, (name, j)


STEPS = [  # B, H, KV, d, window, sinks
    (1, 1, 1, 64, 1, 0), (2, 4, 2, 128, 7, 1), (3, 6, 1, 64, 64, 4), (2, 8, 8, 128, 65, 0), (2, 16, 1, 64, 300, 16),
    (1, 40, 2, 128, 130, 3), (4, 16, 4, 128, 1024, 4), (1, 4, 1, 64, 5000, 4), (1, 2, 2, 128, 3, 20),
]


@pytest.mark.parametrize("B,H,KV,d,window,sinks", STEPS)
def test_step(B, H, KV, d, window, sinks):
    """Positions in the sinks, in a part-filled and in a full ring; slots not yet stored hold NaN."""
    g = torch.Generator().manual_seed(window)
    slots = window + sinks
    for at in (0, 1, sinks, sinks + window // 2, slots - 1, slots, 3 * slots + 5):
        q, k, v = (torch.randn(B, n, d, generator=g).to(BF16) for n in (H, KV, KV))
        kc, vc = (torch.randn(B, KV, slots, d, generator=g).to(BF16) for _ in range(2))
        pos = torch.tensor([max(0, at - b) for b in range(B)], dtype=torch.int32)
        for b in range(B):
            kc[b, :, int(pos[b]):] = float("nan")
            vc[b, :, int(pos[b]):] = float("nan")
        if at >= slots:
            kc, vc = (torch.randn(B, KV, slots, d, generator=g).to(BF16) for _ in range(2))
        want, tol, kw, vw = ref.swa_step(q, k, v, kc, vc, pos, sinks)
        c, y = [t.cuda() for t in (q, k, v, kc, vc, pos)], nan((B, H, d))
        assert ssm.swa_step(*c, sinks=sinks, y=y) is y
        ref.assert_close(y, want, tol, ("y", at))
        same = [torch.equal(a.cpu().view(torch.int16), b.view(torch.int16)) for a, b in ((c[3], kw), (c[4], vw))]
        assert all(same), at


def test_step_leaves_rows_without_a_token():
    q, k, v = (torch.randn(3, n, 64, device="cuda").to(BF16) for n in (4, 2, 2))
    kc, vc = (torch.randn(3, 2, 40, 64, device="cuda").to(BF16) for _ in range(2))
    before = kc.clone(), vc.clone()
    y = ssm.swa_step(q, k, v, kc, vc, torch.tensor([5, -1, 90], dtype=torch.int32, device="cuda"), sinks=4, y=nan(q.shape))
    assert not y[1].any() and y[0].any() and y[2].any()
    assert torch.equal(kc[1], before[0][1]) and torch.equal(vc[1], before[1][1]) and not torch.equal(kc, before[0])


@pytest.mark.parametrize("window,sinks,d", [(10, 3, 64), (64, 0, 128), (33, 5, 64), (200, 4, 128)])
def test_prompt_then_steps_matches_the_whole_sequence(window, sinks, d):
    B, L, H, KV = 3, 120, 4, 2
    q, k, v, _ = make(B, L, H, KV, d, 9)
    lengths = torch.tensor([100, 2, 57], dtype=torch.int32)
    want, tol = ref.swa(q, k, v, window, sinks)
    kc, vc = (nan((B, KV, window + sinks, d)) for _ in range(2))
    ssm.swa_fill(k.cuda(), v.cuda(), kc, vc, sinks=sinks, lengths=lengths.cuda())
    pos = lengths.clone()
    rows = torch.arange(B)
    for _ in range(20):
        p = pos.long()
        y = ssm.swa_step(q[rows, p].cuda(), k[rows, p].cuda(), v[rows, p].cuda(), kc, vc, pos.cuda(), sinks=sinks)
        ref.assert_close(y, want["y"][rows, p], tol["y"][rows, p], "y")
        pos += 1


def test_fill_leaves_other_slots():
    k, v = (torch.randn(2, 6, 1, 64, device="cuda").to(BF16) for _ in range(2))
    kc, vc = (torch.zeros(2, 1, 12, 64, device="cuda", dtype=BF16) for _ in range(2))
    ssm.swa_fill(k, v, kc, vc, sinks=2, lengths=torch.tensor([0, 5], dtype=torch.int32, device="cuda"))
    assert not kc[0].any() and torch.equal(kc[1, 0, :5], k[1, :5, 0]) and not kc[1, 0, 5:].any()
    assert torch.equal(vc[1, 0, :5], v[1, :5, 0])


def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph():
    B, L, H, KV, d = 2, 600, 4, 2, 64
    q, k, v, dy = (t.cuda() for t in make(B, L, H, KV, d, 10))
    kc, vc = (torch.randn(B, KV, 2004, d, device="cuda").to(BF16) for _ in range(2))
    pos = torch.tensor([700, 5000], dtype=torch.int32, device="cuda")
    kw = dict(window=150, sinks=4)

    def all_of(stream=None):
        y, lse = ssm.swa_fwd(q, k, v, **kw, stream=stream)
        step = ssm.swa_step(q[:, 0], k[:, 0], v[:, 0], kc, vc, pos, sinks=4, stream=stream)
        return (y, lse, step) + ssm.swa_bwd(q, k, v, y, lse, dy, **kw, stream=stream)

    first = [t.clone() for t in all_of()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = all_of(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = all_of()
    for _ in range(3):
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, held))
        assert all(torch.equal(a, b) for a, b in zip(first, all_of()))


def test_offsets_past_32_bits():
    """A fused projection and a cache past 2^31 elements: their last rows against dense copies."""
    wide = torch.zeros(2, 520, 2 ** 21 + 64, device="cuda", dtype=BF16)
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (wide[..., i * 64:(i + 1) * 64].unflatten(-1, (1, 64)) for i in range(3))
    for t in (q, k, v):
        t.copy_(torch.randn(2, 520, 1, 64, device="cuda", generator=g).to(BF16))
    dense = [t.contiguous() for t in (q, k, v)]
    y, lse = ssm.swa_fwd(q, k, v, window=100, sinks=2)
    y2, lse2 = ssm.swa_fwd(*dense, window=100, sinks=2)
    assert torch.equal(y, y2) and torch.equal(lse, lse2)
    del wide, q, k, v
    kc, vc = (torch.randn(70, 8, 32768, 128, device="cuda", dtype=BF16) for _ in range(2))
    q, k, v = (torch.randn(70, n, 128, device="cuda", dtype=BF16) for n in (8, 8, 8))
    pos = torch.full((70,), 40000, dtype=torch.int32, device="cuda")
    tail = [t[-1:].clone() for t in (q, k, v, kc, vc, pos)]
    y = ssm.swa_step(q, k, v, kc, vc, pos)
    y2 = ssm.swa_step(*tail)
    ref.assert_close(y[-1:], ref.f64(y2), 2.0 ** -7 * (y2.float().abs().cpu().double().numpy() + 0.05), "y")
    assert torch.equal(kc[-1:], tail[3]) and torch.equal(vc[-1:], tail[4])


def test_nan_queries_give_nan_alone():
    q, k, v, _ = make(1, 100, 2, 1, 64, 12)
    clean, _ = ssm.swa_fwd(q.cuda(), k.cuda(), v.cuda(), window=30, sinks=1)
    q[0, 40, 1, 5] = float("nan")
    y, _ = ssm.swa_fwd(q.cuda(), k.cuda(), v.cuda(), window=30, sinks=1)
    bad = torch.isnan(y.float()).cpu()
    assert bad[0, 40, 1].all() and int(bad.sum()) == 64 and torch.equal(y.cpu()[~bad], clean.cpu()[~bad])
    kc, vc = (torch.randn(1, 1, 400, 64, device="cuda").to(BF16) for _ in range(2))
    pos = torch.tensor([900], dtype=torch.int32, device="cuda")
    y = ssm.swa_step(q[:, 40].cuda(), k[:, 40].cuda(), v[:, 40].cuda(), kc, vc, pos)
    assert torch.isnan(y[0, 1].float()).all() and not torch.isnan(y[0, 0].float()).any()


@pytest.mark.parametrize("d", [64, 128])
def test_slots_past_2_31_elements_of_one_head(d):
    """One head's cache of more than 2^31 elements, its keys far from the query but for the last 64: the token takes
    its slot at the end of a part-filled and of a full ring, and no other slot changes."""
    slots, sinks, tail = 2 ** 31 // d + 100, 4, 64
    kc, vc = (torch.full((1, 1, slots, d), -16.0, dtype=BF16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(d)
    kc[0, 0, -tail:], vc[0, 0, -tail:] = (torch.randn(tail, d, generator=g).to(BF16).cuda() for _ in range(2))
    q = torch.ones(1, 1, d, dtype=BF16)
    for at in (slots - 3, 2 * slots - sinks - 2):
        k, v = (torch.randn(1, 1, d, generator=g).to(BF16) for _ in range(2))
        slot = at if at < slots else at - (slots - sinks)
        count = min(at + 1, slots) - (slots - tail)   # of the last 64 slots
        kt, vt = kc[0, 0, -tail:].cpu(), vc[0, 0, -tail:].cpu()
        kt[slot - slots], vt[slot - slots] = k[0, 0], v[0, 0]
        # The other keys' scores are -16 sqrt(d): 2^25 weights of e^-128 are nothing beside the tail's.
        s = (ref.f64(kt[:count]) @ ref.f64(q[0, 0])) / d ** 0.5
        w = np.exp(s) / np.exp(s).sum()
        want, size = w @ ref.f64(vt[:count]), w @ np.abs(ref.f64(vt[:count]))
        y = ssm.swa_step(q.cuda(), k.cuda(), v.cuda(), kc, vc, torch.tensor([at], dtype=torch.int32, device="cuda"), sinks=sinks)
        ref.assert_close(y[0, 0], want, ref.U * np.abs(want) + (ref.U + 2.0 ** -14) * size, ("y", at))
        assert torch.equal(kc[0, 0, -tail:].cpu(), kt) and torch.equal(vc[0, 0, -tail:].cpu(), vt), at
        for cache in (kc, vc):
            assert all(bool((part == -16).all()) for part in cache[0, 0, :-tail].split(1 << 20))


def test_many_sinks():
    """More (sink, later query) pairs than workgroups of their own: each takes a longer turn."""
    B, L, H, window, sinks = 16, 2600, 8, 40, 640
    q, k, v, dy = make(B, L, H, 1, 64, 14)
    c, kw = [t.cuda() for t in (q, k, v)], dict(window=window, sinks=sinks)
    y, lse = ssm.swa_fwd(*c, **kw)
    got = dict(zip(("dq", "dk", "dv"), ssm.swa_bwd(*c, y, lse, dy.cuda(), **kw)))
    row = slice(B - 1, B)
    want, tol = ref.swa(q[row], k[row], v[row], window, sinks, dy=dy[row])
    for n, t in got.items():
        ref.assert_close(t[row], want[n], tol[n], n)


def test_fill_past_2_32_pieces():
    """Caches of more 16-byte pieces than a launch has threads: the prompts of the last rows arrive."""
    B, KV, d, slots, L = 16, 8, 128, 2 ** 21 + 8, 9
    k, v = (torch.randn(B, L, KV, d, device="cuda").to(BF16) for _ in range(2))
    kc, vc = (torch.empty(B, KV, slots, d, dtype=BF16, device="cuda") for _ in range(2))
    for cache in (kc, vc):
        cache[:, :, :L + 1].zero_()
    ssm.swa_fill(k, v, kc, vc, sinks=4)
    for cache, new in ((kc, k), (vc, v)):
        assert torch.equal(cache[:, :, :L], new.transpose(1, 2)) and not cache[:, :, L].any()
    del kc, vc, cache
    torch.cuda.empty_cache()   # 128 GiB


@pytest.mark.parametrize("d,window,sinks", [(64, 60, 2), (128, 60, 2), (64, 33, 0), (128, 500, 3), (64, 20, 70)])
@pytest.mark.parametrize("lengths", [None, [400, 261]])
def test_gradients_of_what_is_not_seen_stay_as_they_were(d, window, sinks, lengths):
    """NaN and infinities in keys, values, queries and gradients reach the rows that see them, or are seen by them, alone."""
    B, L, H, KV = 2, 400, 4, 2
    q, k, v, dy = make(B, L, H, KV, d, 15)
    n = torch.tensor(lengths or [L, L])
    kw = dict(window=window, sinks=sinks, lengths=None if lengths is None else n.to(torch.int32).cuda())
    see = torch.from_numpy(np.stack([np.pad(ref.visible(m, window, sinks, m), ((0, L - m), (0, L - m))) for m in n.tolist()]))

    def run(q, k, v, dy):
        c = [t.cuda() for t in (q, k, v)]
        y, lse = ssm.swa_fwd(*c, **kw)
        out = {name: nan(t.shape) for name, t in (("dq", q), ("dk", k), ("dv", v))}
        ssm.swa_bwd(*c, y, lse, dy.cuda(), **kw, out=out)
        return {name: t.cpu() for name, t in out.items()}

    clean = run(q, k, v, dy)
    head, group = torch.arange(H), H // KV
    for what, at, bad in (("k", 100, "nan"), ("k", 100, "inf"), ("v", 250, "-inf"), ("q", 130, "nan"), ("q", 255, "inf"),
                          ("dy", 130, "inf"), ("dy", 7, "nan")):
        t = dict(q=q.clone(), k=k.clone(), v=v.clone(), dy=dy.clone())
        h = 1 if what in ("k", "v") else 2              # a head of its own kind: key head 1, or its first query head
        t[what][:, at, h, 5] = float(bad)
        got = run(**t)
        # Queries whose weights or gradients are not finite: those that see the key, or the one itself.
        hit = torch.zeros(B, L, H, dtype=torch.bool)
        if what in ("k", "v"):
            hit[:] = see[:, :, at, None] & (head // group == h)
        else:
            hit[:, at, h] = at < n
        seen_by_hit = torch.stack([(see[:, :, :, None] & hit[:, :, None, c * group:(c + 1) * group]).any(-1).any(1)
                                   for c in range(KV)], -1)             # keys that such a query sees
        assert torch.equal(got["dq"][~hit], clean["dq"][~hit]), (what, bad)
        assert torch.equal(got["dk"][~seen_by_hit], clean["dk"][~seen_by_hit]), (what, bad)
        touched = seen_by_hit if what != "v" else torch.zeros_like(seen_by_hit)   # values do not reach dv
        assert torch.equal(got["dv"][~touched], clean["dv"][~touched]), (what, bad)
        bad_dq, bad_dk, bad_dv = (~torch.isfinite(got[name].float()) for name in ("dq", "dk", "dv"))
        if bad == "nan" and what != "v":
            assert bad_dq[hit].all() and bad_dk[seen_by_hit].all()
        if what == "dy":                                 # dv gets p times it in its element alone
            assert bad_dv[seen_by_hit][:, 5].all() and not bad_dv[..., :5].any() and not bad_dv[..., 6:].any()
            want = torch.isnan if bad == "nan" else lambda x: x == float("inf")
            assert want(got["dv"][seen_by_hit][:, 5].float()).all()
        elif bad == "nan":
            assert bad_dv[seen_by_hit].all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at,slot", [(9, 9), (9, 4), (200, 100), (300, 137), (273, 136)])
def test_an_infinity_among_a_steps_values_stays_one(d, at, slot):
    """In the token's own value or a stored one, last of a tile or not: its element alone, and not a NaN."""
    window, sinks = 134, 3
    g = torch.Generator().manual_seed(at)
    q, k, v = (torch.randn(1, n, d, generator=g).to(BF16).cuda() for n in (4, 2, 2))
    kc, vc = (torch.randn(1, 2, window + sinks, d, generator=g).to(BF16).cuda() for _ in range(2))
    own = at if at < sinks else sinks + (at - sinks) % window
    slot = min(slot, window + sinks - 1)
    pos = torch.tensor([at], dtype=torch.int32, device="cuda")
    clean = ssm.swa_step(q, k, v, kc.clone(), vc.clone(), pos, sinks=sinks)
    vc[0, 1, slot, 5] = float("-inf")
    if slot == own:
        v[0, 1, 5] = float("-inf")
    y = ssm.swa_step(q, k, v, kc, vc, pos, sinks=sinks)
    assert bool((y[0, 2:, 5] == float("-inf")).all())
    y[0, 2:, 5] = clean[0, 2:, 5]
    assert torch.equal(y, clean)
