"""Residual addition with RMS norm (plain, 8-bit, backward) against float64."""
import numpy as np
import pytest
import torch

import block_reference as ref
import state_space_model_ssm_amd as ssm

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(rows, dim, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x, res, dy, dres = ((torch.randn(rows, dim, generator=g) * s).to(dtype) for s in (1.0, 2.0, 1.0, 1.0))
    return x, res, 1 + 0.2 * torch.randn(dim, generator=g), dy, dres


def nan(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


SIZES = [(1, 1), (3, 2), (5, 7), (2, 64), (33, 65), (4, 128), (7, 255), (3, 256), (1, 512), (130, 520), (9, 1000),
         (2, 1024), (70, 1537), (3, 2048), (5, 4104), (2, 5120), (3, 8192), (2, 8200), (1, 16384), (2, 20001),
         (1030, 96)]


@pytest.mark.parametrize("rows,dim", SIZES)
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
def test_forward(rows, dim, dtype, out):
    x, res, w, _, _ = make(rows, dim, dtype, rows + dim)
    y, s = nan((rows, dim), out), nan((rows, dim), dtype)
    got = ssm.rms_add_fwd(x.cuda(), w.cuda(), res.cuda(), out_dtype=out, y=y, residual_out=s)
    assert got[0] is y and got[1] is s
    want, total = ref.rms(x, w, res)
    ref.assert_close(y, want, ref.storage_tol(want, out), "y")
    ref.assert_close(s, total, ref.storage_tol(total, dtype), "s")
    y, s = ssm.rms_add_fwd(x.cuda(), w.cuda(), out_dtype=out, eps=0.1)
    want, _ = ref.rms(x, w, eps=0.1)
    ref.assert_close(y, want, ref.storage_tol(want, out), "y without residual")
    assert torch.equal(s.cpu(), x)


@pytest.mark.parametrize("rows,dim", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward(rows, dim, dtype):
    _, s, w, dy, dres = make(rows, dim, dtype, rows * 3 + dim)
    dx, dw = nan((rows, dim), dtype), nan((dim,), F32)
    ssm.rms_add_bwd(dy.cuda(), s.cuda(), w.cuda(), dres=dres.cuda(), dx=dx, dw=dw)
    want, want_w, size = ref.rms_bwd(dy, s, w, dres)
    ref.assert_close(dx, want, ref.storage_tol(want, dtype), "dx")
    ref.assert_close(dw, want_w, ref.storage_tol(want_w, F32, size), "dw")
    dx, none = ssm.rms_add_bwd(dy.cuda(), s.cuda(), w.cuda(), return_dw=False, eps=0.1)
    want, _, _ = ref.rms_bwd(dy, s, w, eps=0.1)
    assert none is None
    ref.assert_close(dx, want, ref.storage_tol(want, dtype), "dx without dres and dw")


def test_backward_against_differences():
    _, s, w, dy, dres = make(3, 70, F32, 1)
    dx, dw = ssm.rms_add_bwd(dy.cuda(), s.cuda(), w.cuda(), dres=dres.cuda(), eps=1e-3)

    def loss(s, w):
        return float((ref.rms(s, w, eps=1e-3)[0] * ref.f64(dy)).sum() + (ref.f64(s) * ref.f64(dres)).sum())

    for k, t in enumerate((dx, dw)):
        for j in np.random.default_rng(k).integers(0, t.numel(), 8):
            at = [[v.double().clone() for v in (s, w)] for _ in range(2)]
            at[0][k].view(-1)[j] += 1e-5
            at[1][k].view(-1)[j] -= 1e-5
            want = (loss(*at[0]) - loss(*at[1])) / 2e-5
            assert abs(float(t.view(-1)[j]) - want) <= 1e-5 * max(1.0, float(t.abs().max())), (k, j)


@pytest.mark.parametrize("rows,dim,group", [(1, 1, 0), (5, 7, 0), (3, 64, 32), (33, 65, 32), (4, 128, 128), (7, 255, 64),
                                            (130, 520, 128), (2, 1024, 0), (70, 1537, 128), (3, 2048, 96),
                                            (2, 5120, 0), (2, 5120, 128), (3, 8200, 128), (1, 20001, 0), (2, 20001, 1024),
                                            (4, 100, 512)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_8_bit_output(rows, dim, group, dtype):
    x, res, w, _, _ = make(rows, dim, dtype, rows + dim)
    width = group if 0 < group < dim else dim
    groups = -(-dim // width)
    q, scale, s = nan((rows, dim), E4M3), nan((rows, groups), F32), nan((rows, dim), dtype)
    ssm.rms_add_q8_fwd(x.cuda(), w.cuda(), res.cuda(), group=group, q=q, scale=scale, residual_out=s)
    want, total = ref.rms(x, w, res)
    ref.assert_close(s, total, ref.storage_tol(total, dtype), "s")
    tops = np.stack([np.abs(want[:, k * width:(k + 1) * width]).max(1) / 448 for k in range(groups)], 1)
    ref.assert_close(scale, tops, 1e-6 * tops, "scale")
    # q is the nearest e4m3 value of y / scale; 1e-6 of its size lets float32 fall on either side of a tie.
    v = want / np.repeat(ref.f64(scale), width, 1)[:, :dim]
    table = ref.e4m3_values()
    got = q.float().cpu().double().numpy()
    near = table[np.abs(table[None] - v.reshape(-1, 1)).argmin(1)].reshape(v.shape) if v.size < 50000 else None
    if near is not None:
        assert np.all(np.abs(got - v) <= np.abs(near - v) + 2e-6 * np.abs(v) + 1e-9)
    assert np.all(np.abs(got - v) <= np.maximum(np.abs(v) / 16, 2.0 ** -10) * (1 + 1e-5))


# Widths about the 16 bytes of a load, and rows that start at any value.
@pytest.mark.parametrize("dim", [3, 4, 5, 8, 9, 15, 17, 63, 66, 257, 1023, 4097, 8191])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_that_start_at_any_value(dim, dtype):
    rows = 5
    x, res, w, dy, dres = make(rows, dim, dtype, dim)

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.flatten()
        return flat[1:].view(t.shape)

    a, b = shifted(x), shifted(res)
    y, s = ssm.rms_add_fwd(a, shifted(w), b, y=shifted(nan((rows, dim), dtype)), residual_out=shifted(nan((rows, dim), dtype)))
    want, total = ref.rms(x, w, res)
    ref.assert_close(s, total, ref.storage_tol(total, dtype), "s")
    ref.assert_close(y, want, ref.storage_tol(want, dtype), "y")
    ssm.rms_add_fwd(a, shifted(w), b, y=a, residual_out=b)  # in place
    assert torch.equal(a, y) and torch.equal(b, s)
    q, scale, _ = ssm.rms_add_q8_fwd(x.cuda(), w.cuda(), res.cuda())
    q2, scale2, s2 = ssm.rms_add_q8_fwd(shifted(x), shifted(w), shifted(res))
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(scale, scale2) and torch.equal(s2, s)
    dx, dw = ssm.rms_add_bwd(shifted(dy), s, shifted(w), dres=shifted(dres), dw=shifted(nan((dim,), F32)))
    aligned = ssm.rms_add_bwd(dy.cuda(), s.clone(), w.cuda(), dres=dres.cuda())
    want, want_w, size = ref.rms_bwd(dy, s.cpu(), w, dres)
    for got in ((dx, dw), aligned):
        ref.assert_close(got[0], want, ref.storage_tol(want, dtype), "dx")
        ref.assert_close(got[1], want_w, ref.storage_tol(want_w, F32, size), "dw")


def test_8_bit_output_of_zeros_and_nan():
    x = torch.randn(4, 256)
    x[1] = 0
    x[2, 130] = float("nan")
    q, scale, _ = ssm.rms_add_q8_fwd(x.cuda(), torch.ones(256).cuda(), group=128)
    assert not q[1].float().any() and not scale[1].any()
    assert torch.isnan(scale[2]).all() and torch.isnan(q[2].float()).all()   # the row's norm is NaN
    assert not torch.isnan(scale[[0, 1, 3]]).any() and not torch.isnan(q[[0, 1, 3]].float()).any()
    w = torch.ones(256)
    w[5] = float("nan")
    q, scale, _ = ssm.rms_add_q8_fwd(x[:1].cuda(), w.cuda(), group=128)
    assert torch.isnan(scale[0, 0]) and not torch.isnan(scale[0, 1])


def test_rows_do_not_meet():
    x, res, w, _, _ = make(6, 300, F32, 3)
    clean, _ = ssm.rms_add_fwd(x.cuda(), w.cuda(), res.cuda())
    x[2, 7], x[4, 100] = float("inf"), float("nan")
    y, _ = ssm.rms_add_fwd(x.cuda(), w.cuda(), res.cuda())
    keep = [0, 1, 3, 5]
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[4]).all() and torch.isnan(y[2, 7])


@pytest.mark.parametrize("dtype,dim", [(BF16, 1024), (F32, 1537)])
def test_in_place(dtype, dim):
    x, res, w, dy, dres = (t.cuda() for t in make(40, dim, dtype, 4))
    y, s = ssm.rms_add_fwd(x, w, res)
    a, b = x.clone(), res.clone()
    ssm.rms_add_fwd(a, w, b, y=a, residual_out=b)
    assert torch.equal(a, y) and torch.equal(b, s)
    a = x.clone()
    q, scale, s2 = ssm.rms_add_q8_fwd(a, w, res, residual_out=a)
    assert s2 is a and torch.equal(a, s)
    dx, _ = ssm.rms_add_bwd(dy, s, w, dres=dres)
    a = dres.clone()
    ssm.rms_add_bwd(dy, s, w, dres=a, dx=a)
    assert torch.equal(a, dx)


def test_unaligned_rows():
    """A tensor that starts at an element, not at a vector: the same values as its aligned copy."""
    for dtype, dim in ((BF16, 1024), (F32, 512)):
        flat = torch.randn(9 * dim + 1, device="cuda").to(dtype)
        x, w = flat[1:].view(9, dim), torch.rand(dim + 1, device="cuda")[1:]
        y, _ = ssm.rms_add_fwd(x, w)
        ref_y = ref.rms(x, w)[0]
        ref.assert_close(y, ref_y, ref.storage_tol(ref_y, dtype), "y")
        dx, dw = ssm.rms_add_bwd(x, x, w)
        want, want_w, size = ref.rms_bwd(x, x, w)
        ref.assert_close(dx, want, ref.storage_tol(want, dtype), "dx")
        ref.assert_close(dw, want_w, ref.storage_tol(want_w, F32, size), "dw")


def test_leading_axes_and_no_rows():
    w = torch.ones(48, device="cuda")
    x = torch.randn(2, 3, 5, 48, device="cuda")
    assert torch.equal(ssm.rms_add_fwd(x, w)[0], ssm.rms_add_fwd(x.view(30, 48), w)[0].view(x.shape))
    assert ssm.rms_add_q8_fwd(x, w, group=32)[1].shape == (2, 3, 5, 2)
    e = torch.empty(0, 48, device="cuda")
    dw = nan((48,), F32)
    assert ssm.rms_add_fwd(e, w, e)[0].shape == (0, 48) and ssm.rms_add_q8_fwd(e, w)[1].shape == (0, 1)
    ssm.rms_add_bwd(e, e, w, dw=dw)
    assert not dw.any()


def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph():
    x, res, w, dy, dres = (t.cuda() for t in make(3000, 640, BF16, 8))

    def all_of(stream=None):
        y, s = ssm.rms_add_fwd(x, w, res, stream=stream)
        q, scale, _ = ssm.rms_add_q8_fwd(x, w, res, group=128, stream=stream)
        return (y, s, q.view(torch.uint8), scale) + ssm.rms_add_bwd(dy, s, w, dres=dres, stream=stream)

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
    rows, dim = 262150, 8200
    x = torch.randn(rows, dim, device="cuda", dtype=BF16)
    w = torch.rand(dim, device="cuda") + 0.5
    y, s = ssm.rms_add_fwd(x, w, x)
    tail = x[-8:].contiguous()
    y2, s2 = ssm.rms_add_fwd(tail, w, tail)
    assert torch.equal(y[-8:], y2) and torch.equal(s[-8:], s2)
    dx, _ = ssm.rms_add_bwd(x, x, w, dres=x, return_dw=False)
    assert torch.equal(dx[-8:], ssm.rms_add_bwd(tail, tail, w, dres=tail, return_dw=False)[0])


def test_8_bit_output_of_tiny_values():
    """Scales far below float32's normal range keep their values' ratios."""
    for dim, group in ((256, 0), (256, 128), (101, 0), (256, 96)):
        w = torch.full((dim,), 1e-36)
        x = torch.randn(3, dim, generator=torch.Generator().manual_seed(dim))
        x[0, 3] = 0
        q, scale, _ = ssm.rms_add_q8_fwd(x.cuda(), w.cuda(), group=group)
        want, _ = ref.rms(x, w)
        got = q.float().cpu().double().numpy() * np.repeat(ref.f64(scale), group or dim, 1)[:, :dim]
        # half a step of e4m3 (2^-4 of a value), and the scale's own step of 2^-149 against about 2^-128
        assert np.all(np.abs(got - want) <= np.abs(want) * (2.0 ** -4 + 2.0 ** -18) + 2.0 ** -10 * np.abs(want).max())


def test_sums_of_long_rows():
    """A row of 2^27 equal values, whose squares take more bits than a sum of them leaves: y is w, dx is 0."""
    dim = 2 ** 27 + 9
    x = torch.full((1, dim), 1.1, dtype=BF16, device="cuda")
    w = torch.ones(dim, device="cuda")
    y, _ = ssm.rms_add_fwd(x, w, out_dtype=F32)
    rstd = 1 / (float(x[0, 0]) ** 2 + 1e-5) ** 0.5
    assert bool(((y.double() - float(x[0, 0]) * rstd).abs() <= 1e-5).all())
    dx, _ = ssm.rms_add_bwd(x, x, w, return_dw=False)
    # dn - n mean(dn n) of equal values: 1 - n^2, times dn and rstd; 1e-5 of dn's part.
    n = float(x[0, 0]) * rstd
    want = rstd * float(x[0, 0]) * (1 - n * n)
    assert bool(((dx.double() - want).abs() <= 1e-5).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_past_2_24(dtype):
    """More narrow rows than a launch has workgroups."""
    rows, dim = 2 ** 24 + 3, 3
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(rows, dim, generator=g, device="cuda").to(dtype)
    w = torch.rand(dim, generator=g, device="cuda") + 0.5
    s = x.double()
    want = s / (s.pow(2).mean(-1, keepdim=True) + 1e-5).sqrt() * w.double()
    top = float(want.abs().max())
    y, _ = ssm.rms_add_fwd(x, w, y=nan((rows, dim), dtype))
    tol = 1e-5 * top + (ref.U * want.abs() if dtype == BF16 else 0.0)
    assert bool(((y.double() - want).abs() <= tol).all())
    q, scale, _ = ssm.rms_add_q8_fwd(x, w, q=nan((rows, dim), E4M3), scale=nan((rows, 1), F32))
    amax = want.abs().amax(-1, keepdim=True)
    assert bool(((scale.double() * 448 - amax).abs() <= 1e-6 * amax).all())
    # Half a step of e4m3: 2^-4 of a value, 2^-10 of the scale near zero.
    err = (q.double() * scale.double() - want).abs()
    assert bool((err <= (want.abs() / 16).maximum(scale.double() * 2.0 ** -10) * (1 + 1e-5) + 1e-6 * amax).all())


def test_dw_of_columns_past_2_28():
    """dw of more columns than a launch of its sum has threads for."""
    dim = 2 ** 28 + 70
    g = torch.Generator(device="cuda").manual_seed(6)
    s, dy = (torch.randn(1, dim, generator=g, device="cuda", dtype=BF16) for _ in range(2))
    w = torch.ones(dim, device="cuda")
    dw = nan((dim,), F32)
    ssm.rms_add_bwd(dy, s, w, dw=dw)
    total = sum(float(part.double().pow(2).sum()) for part in s[0].split(1 << 24))
    rstd = 1 / (total / dim + 1e-5) ** 0.5
    for lo in range(0, dim, 1 << 24):
        want = dy[0, lo:lo + (1 << 24)].double() * s[0, lo:lo + (1 << 24)].double() * rstd
        assert bool(((dw[lo:lo + (1 << 24)].double() - want).abs() <= 1e-5 * want.abs().max()).all()), lo


@pytest.mark.parametrize("dtype,dim", [(BF16, 1024), (F32, 1537), (F32, 3), (F32, 8200)])
def test_in_place_without_a_residual_keeps_the_sum(dtype, dim):
    x, _, w, _, _ = (t.cuda() for t in make(6, dim, dtype, 9))
    want, same = ssm.rms_add_fwd(x, w)
    assert same is x
    a = x.clone()
    y, s = ssm.rms_add_fwd(a, w, y=a)
    assert y is a and torch.equal(y, want) and torch.equal(s, x)
