"""Plain float64 implementations of libssm_block's operators, in numpy, for
the tests.  They take torch tensors (widened exactly) and share no code with
the kernels.  Where an output's tolerance depends on the data, the bound is
computed here too, from the roundings the kernels make."""
import numpy as np
import torch

# Largest relative error of one rounding to bfloat16 (8 significant bits).
U = 2.0 ** -8
# What underflow may drop from a sum of a few thousand terms of order 1 to 2^6.
TINY = 2.0 ** -126 * 2 ** 18


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def glr(x, rec, inp, A, h0=None, reset=None):
    """h (batch, L, dim), and the gates needed by the gradient."""
    x, rec, inp, A = f64(x), f64(rec), f64(inp), f64(A)
    r, i = sigmoid(rec), sigmoid(inp)
    la = A * r
    a, b = np.exp(la), np.sqrt(-np.expm1(2 * la))
    keep = np.ones(x.shape[:2]) if reset is None else (f64(reset) == 0).astype(float)
    prev = np.zeros((x.shape[0], x.shape[2])) if h0 is None else f64(h0)
    h, before = np.zeros_like(x), np.zeros_like(x)
    for t in range(x.shape[1]):
        before[:, t] = prev * keep[:, t, None]
        prev = a[:, t] * before[:, t] + b[:, t] * i[:, t] * x[:, t]
        h[:, t] = prev
    return h, prev, dict(x=x, r=r, i=i, a=a, b=b, A=A, before=before, keep=keep)


def glr_bwd(x, rec, inp, A, dy, h0=None, reset=None, dh_last=None):
    _, _, s = glr(x, rec, inp, A, h0, reset)
    dy = f64(dy)
    carry = np.zeros(dy.shape[::2]) if dh_last is None else f64(dh_last).copy()
    g = np.zeros_like(dy)
    for t in range(dy.shape[1] - 1, -1, -1):
        g[:, t] = dy[:, t] + carry
        carry = s["a"][:, t] * g[:, t] * s["keep"][:, t, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        slope = np.where(s["b"] > 0, s["a"] ** 2 / s["b"], 0.0)
    w = g * (s["a"] * s["before"] - slope * s["i"] * s["x"])
    out = {"dx": g * s["b"] * s["i"], "drec": w * s["A"] * s["r"] * (1 - s["r"]),
           "dinp": g * s["b"] * s["x"] * s["i"] * (1 - s["i"]), "dA": (w * s["r"]).sum((0, 1)), "dh0": carry}
    # The terms of each sum, for the tolerance of what cancels.
    size = {"dA": np.abs(w * s["r"]).sum((0, 1))}
    return out, size


def rms(x, w, residual=None, eps=1e-5):
    s = f64(x) + (0.0 if residual is None else f64(residual))
    n = s / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    return n * f64(w), s


def rms_bwd(dy, s, w, dres=None, eps=1e-5):
    dy, s, w = f64(dy), f64(s), f64(w)
    rstd = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    n, dn = s * rstd, dy * w
    dx = rstd * (dn - n * (dn * n).mean(-1, keepdims=True)) + (0.0 if dres is None else f64(dres))
    return dx, (dy * n).reshape(-1, n.shape[-1]).sum(0), np.abs(dy * n).reshape(-1, n.shape[-1]).sum(0)


def e4m3_values():
    """Every finite value of the 8-bit format, ascending."""
    b = np.arange(256)
    s, e, m = b >> 7, (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0)) * np.where(s == 1, -1, 1)
    return np.unique(v[(b & 127) != 127])


def visible(L, window, sinks, n):
    t = np.arange(L)
    gap = t[:, None] - t[None]
    return (gap >= 0) & ((gap < window) | (t[None] < sinks)) & (t[:, None] < n) & (t[None] < n)


def swa(q, k, v, window, sinks, lengths=None, scale=None, dy=None):
    """Outputs and, with dy, gradients; each with a bound of its error.

    The bounds follow the kernels' roundings: products of bfloat16 values are
    exact in float32 sums; p (forward, dv) and ds (dq, dk) are rounded to
    bfloat16 before their products, outputs when they are stored; dy.y reads
    the rounded y.  2^-14 of the terms' sizes stands for the float32 sums and
    the exponentials (scores up to about 30 in size, 2^-24 each, over sums of
    up to 2^8 terms)."""
    q, k, v, dy = f64(q), f64(k), f64(v), f64(dy)
    B, L, H, d = q.shape
    group = H // k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    small = 2.0 ** -14
    val = {"y": np.zeros_like(q), "lse": np.full((B, H, L), -np.inf)}
    tol = {"y": np.zeros_like(q)}
    if dy is not None:
        for name, t in (("dq", q), ("dk", k), ("dv", v)):
            val[name], tol[name] = np.zeros_like(t), np.zeros_like(t)
    for b in range(B):
        n = L if lengths is None else min(max(int(lengths[b]), 0), L)
        if n == 0:
            continue
        see = visible(n, window, sinks, n)
        for h in range(H):
            c = h // group
            Q, K, V = q[b, :n, h], k[b, :n, c], v[b, :n, c]
            s = np.where(see, Q @ K.T * scale, -np.inf)
            top = s.max(1, keepdims=True)
            e = np.exp(s - top)
            total = e.sum(1, keepdims=True)
            p = e / total
            o, oa = p @ V, p @ np.abs(V)
            val["y"][b, :n, h], tol["y"][b, :n, h] = o, U * np.abs(o) + (U + small) * oa
            val["lse"][b, h, :n] = (top + np.log(total))[:, 0]
            if dy is None:
                continue
            G = dy[b, :n, h]
            dp = G @ V.T
            delta = (G * o).sum(1, keepdims=True)
            ds = p * (dp - delta)
            # error of delta from the rounded y, and of p through lse
            ds_err = (U + small) * np.abs(ds) + p * ((tol["y"][b, :n, h] * np.abs(G)).sum(1, keepdims=True)
                                                     + small * (np.abs(G) @ np.abs(V).T))
            val["dq"][b, :n, h] = ds @ K * scale
            tol["dq"][b, :n, h] = ds_err @ np.abs(K) * abs(scale)
            val["dk"][b, :n, c] += ds.T @ Q * scale
            tol["dk"][b, :n, c] += ds_err.T @ np.abs(Q) * abs(scale)
            val["dv"][b, :n, c] += p.T @ G
            tol["dv"][b, :n, c] += (U + small) * (p.T @ np.abs(G))
    for name in ("dq", "dk", "dv"):
        if name in val:
            tol[name] += U * np.abs(val[name]) + TINY   # a weight below float32's normal range counts as 0
    return val, tol


def swa_step(q, k, v, kc, vc, pos, sinks, scale=None):
    """y with its bound, and the caches after the step (as the stored values)."""
    kc, vc = kc.clone(), vc.clone()
    B, H, d = q.shape
    nkv, slots = kc.shape[1], kc.shape[2]
    scale = d ** -0.5 if scale is None else scale
    y, tol = np.zeros((B, H, d)), np.zeros((B, H, d))
    for b in range(B):
        p = int(pos[b])
        if p < 0:
            continue
        slot = p if p < sinks else sinks + (p - sinks) % (slots - sinks)
        kc[b, :, slot], vc[b, :, slot] = k[b], v[b]
        m = min(p + 1, slots)
        for h in range(H):
            c = h // (H // nkv)
            s = f64(kc[b, c, :m]) @ f64(q[b, h]) * scale
            e = np.exp(s - s.max())
            w, V = e / e.sum(), f64(vc[b, c, :m])
            y[b, h] = w @ V
            tol[b, h] = U * np.abs(y[b, h]) + (U + 2.0 ** -14) * (w @ np.abs(V))
    return y, tol, kc, vc


def assert_close(got, want, tol, what):
    """Elementwise |got - want| <= tol, with NaN only where want has it."""
    got = got.detach().cpu().double().numpy() if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if got.size == 0:
        return
    bad = np.isnan(got) | ((np.abs(got - want) > tol) & (got != want))
    assert not bad.any(), (what, int(bad.sum()), got.size, np.argwhere(bad)[:4].tolist(),
                           got[bad][:4].tolist(), want[bad][:4].tolist(), np.broadcast_to(tol, got.shape)[bad][:4].tolist())


def storage_tol(want, dtype, size=None):
    """Tolerance of a float32 computation stored in `dtype`: 1e-5 of the
    largest value (or 2^-18 of the terms' sizes), plus one rounding."""
    base = 1e-5 * (np.abs(want).max() if want.size else 0.0) if size is None else 2.0 ** -18 * size
    return base + (U * np.abs(want) if dtype == torch.bfloat16 else 0.0)
