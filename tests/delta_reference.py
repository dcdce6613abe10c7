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
