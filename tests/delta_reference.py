"""Plain float64 implementations of libssm_delta's operators, in torch on the
CPU, for the tests.  They share no code with the kernels."""
import torch

# Largest relative error of one rounding to bfloat16 (8 significant bits).
U = 2.0 ** -8


def f64(t):
    return None if t is None else t.detach().cpu().double()


def gdr(q, k, v, g, beta, h0=None, lengths=None, scale=None):
    """(y, h_last, states before every 64th token, sizes), token by token, of
    float64 tensors (differentiable).  sizes: per token and value element the
    sum of |S||q| scale, what y's terms add up to at most."""
    B, L, H, V = v.shape
    share = H // q.shape[2]
    scale = q.shape[3] ** -0.5 if scale is None else scale
    ys, last, states, sizes = [], [], [], []
    for b in range(B):
        n = L if lengths is None else min(max(int(lengths[b]), 0), L)
        S = torch.zeros(H, V, q.shape[3], dtype=torch.float64) if h0 is None else h0[b]
        row, before, size = [], [], []
        for t in range(n):
            if t % 64 == 0:
                before.append(S)
            kt, qt = (x[b, t].repeat_interleave(share, 0) for x in (k, q))
            S = torch.exp(g[b, t])[:, None, None] * S
            u = beta[b, t][:, None] * (v[b, t] - (S * kt[:, None]).sum(-1))
            S = S + u[:, :, None] * kt[:, None]
            row.append(scale * (S * qt[:, None]).sum(-1))
            size.append(abs(scale) * (S.detach().abs() * qt.detach().abs()[:, None]).sum(-1))
        row += [torch.zeros(H, V, dtype=torch.float64)] * (L - n)
        size += [torch.zeros(H, V, dtype=torch.float64)] * (L - n)
        ys.append(torch.stack(row) if row else torch.zeros(0, H, V, dtype=torch.float64))
        sizes.append(torch.stack(size) if size else torch.zeros(0, H, V, dtype=torch.float64))
        last.append(S)
        states.append(before)
    return torch.stack(ys), torch.stack(last), states, torch.stack(sizes)


def gdr_bwd(q, k, v, g, beta, dy, h0=None, lengths=None, scale=None, dh_last=None):
    """Gradients by the reverse recurrence, and sizes: what the terms of each
    add up to at most, by norms (per token and head; of dg over the rest of
    the token's block of 64, whose products the kernels sum)."""
    B, L, H, V = v.shape
    K, share = q.shape[3], H // q.shape[2]
    scale = K ** -0.5 if scale is None else scale
    zero = torch.zeros(B, H, V, K, dtype=torch.float64)
    grads = {n: torch.zeros_like(t) for n, t in zip(("dq", "dk", "dv", "dg", "dbeta"), (q, k, v, g, beta))}
    sizes = {n: torch.zeros(B, L, H, dtype=torch.float64) for n in grads}
    grads["dh0"] = zero.clone()
    for b in range(B):
        n = L if lengths is None else min(max(int(lengths[b]), 0), L)
        S, past = zero[b] if h0 is None else h0[b], []
        for t in range(n):
            kt, a = k[b, t].repeat_interleave(share, 0), torch.exp(g[b, t])[:, None]
            seen = (S * kt[:, None]).sum(-1)
            rest = v[b, t] - a * seen
            u = beta[b, t][:, None] * rest
            past.append((S, seen, rest, u))
            S = a[:, :, None] * S + u[:, :, None] * kt[:, None]
        dS = zero[b] if dh_last is None else dh_last[b]
        after, run = S, torch.zeros(H, dtype=torch.float64)
        for t in range(n - 1, -1, -1):
            S, seen, rest, u = past[t]
            kt, qt = (x[b, t].repeat_interleave(share, 0) for x in (k, q))
            a, y = torch.exp(g[b, t])[:, None], dy[b, t]
            if t % 64 == 63 or t == n - 1:
                run = (after.flatten(1).norm(dim=1) * dS.flatten(1).norm(dim=1))
            dS = dS + scale * y[:, :, None] * qt[:, None]
            e = (dS * kt[:, None]).sum(-1)
            dv = beta[b, t][:, None] * e
            dq = scale * (after * y[:, :, None]).sum(1)
            write, erase = (dS * u[:, :, None]).sum(1), a * (S * dv[:, :, None]).sum(1)
            grads["dq"][b, t] += dq.unflatten(0, (-1, share)).sum(1)
            grads["dk"][b, t] += (write - erase).unflatten(0, (-1, share)).sum(1)
            grads["dv"][b, t], grads["dbeta"][b, t] = dv, (e * rest).sum(-1)
            grads["dg"][b, t] = a[:, 0] * ((dS * S).sum((1, 2)) - (dv * seen).sum(-1))
            nS, ndS = (x.flatten(1).norm(dim=1) for x in (after, dS))
            nb = S.flatten(1).norm(dim=1)
            nq, nk, ny, nu, nv = (x.norm(dim=-1) for x in (qt, kt, y, u, dv))
            sizes["dq"][b, t] = abs(scale) * ny * nS
            sizes["dk"][b, t] = nu * ndS + a[:, 0] * nv * nb
            sizes["dv"][b, t] = beta[b, t].abs() * ndS * nk
            sizes["dbeta"][b, t] = ndS * nk * (v[b, t].norm(dim=-1) + a[:, 0] * nb * nk)
            run = run + nq * sizes["dq"][b, t] + nk * sizes["dk"][b, t]
            sizes["dg"][b, t] = run
            dS = a[:, :, None] * (dS - dv[:, :, None] * kt[:, None])
            after = S
        grads["dh0"][b] = dS
    return grads, sizes


def qk_norm(x, w, inv_freq, pos, eps, neighbours):
    """One of q and k, (batch, L, heads, d) float64; differentiable."""
    n = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * (1.0 if w is None else w)
    if inv_freq is None:
        return n
    half = inv_freq.shape[0]
    angle = (pos.double()[..., None] * inv_freq.double())[:, :, None]
    a = n[..., 0:2 * half:2] if neighbours else n[..., :half]
    b = n[..., 1:2 * half:2] if neighbours else n[..., half:2 * half]
    c, s = angle.cos(), angle.sin()
    a, b = a * c - b * s, b * c + a * s
    turned = torch.stack([a, b], -1).flatten(-2) if neighbours else torch.cat([a, b], -1)
    return torch.cat([turned, n[..., 2 * half:]], -1)


E4M3 = torch.tensor([[m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for m in range(8)] for e in range(16)],
                    dtype=torch.float64).flatten()[:127]


def to_e4m3(x):
    """Values within +-448 rounded to the nearest of the format, ties to the even one, by its table."""
    hi = torch.searchsorted(E4M3, x.abs().contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = E4M3[hi] - x.abs(), x.abs() - E4M3[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.sign(x) * E4M3[code]


class Q8Cache:
    """An 8-bit cache by the definition: every position's key and value, and what a query would be given of them."""

    def __init__(self, batch, nkv, window, d, sinks):
        self.window, self.sinks = window, sinks
        self.rows = [([], []) for _ in range(batch)]     # per row: keys and values, (nkv, d) per position

    def held(self, b, t, pos):
        """(positions, nkv, d) that position `pos` sees, t = 0 for keys: blocks that were whole before it in 8 bits."""
        x = torch.stack(self.rows[b][t]).double()
        block = (pos - self.sinks) // 64 if pos >= self.sinks else 0
        for n in range(block):
            at = slice(self.sinks + 64 * n, self.sinks + 64 * n + 64)
            block32 = x[at].float()   # scales are float32, and so are the quotients
            scale = block32.abs().amax((0, 2), keepdim=True) / 448
            x[at] = to_e4m3((block32 / torch.where(scale > 0, scale, 1.0)).clamp(-448, 448).double()) * scale.double()
        seen = [j for j in range(pos + 1) if j < self.sinks or pos - j < self.window]
        return x[seen]


def close(got, want, tol, what):
    """Elementwise |got - want| <= tol; NaN nowhere."""
    got, want = f64(got), f64(want)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        at = bad.nonzero()[:4].tolist()
        off = (got - want).abs().nan_to_num(float("inf"))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, by up to {float(off.max()):.3g} "
                             f"(allowed there {float(torch.as_tensor(tol).expand_as(bad)[bad].max()):.3g}), at {at}: "
                             f"{got[bad][:4].tolist()} for {want[bad][:4].tolist()}")
