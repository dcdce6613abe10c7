"""Work of the hybrid-block operators: gated linear recurrence, residual add
with RMS norm, and sliding-window attention with sinks.

Every case is one call (or, for "train", the forward with its backward) on
data that a model's program holds at that point.  ``run`` computes it with
elementary torch operations in float32, or through the library's entry points
when ``own`` is set; ``exact`` computes it from the definitions in float64.

Definitions (s() is the logistic function):
  glr   r = s(rec), i = s(inp), a = exp(A r), b = sqrt(1 - a^2)
        h_t = a_t h_{t-1} + b_t i_t x_t   (h_{t-1} counts as 0 where reset_t)
  rms   s = x + residual, y = s / sqrt(mean(s^2) + eps) * w; "q8" stores y in
        e4m3 floats with one float32 scale, amax / 448, per row or per group
  swa   query t sees key j when j <= t and (t - j < window or j < sinks), both
        within the row's length; softmax of scale * q.k over those keys; a
        query that sees no key gives zeros
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # One token of 64 sequences through a recurrent layer: latency.
        dict(name="glr_step", op="glr", dir="step", dtype="bf16", batch=64, seqlen=1, dim=5120, resets=False),
        # One long prompt of odd length, few channels: the time axis has to be split.
        dict(name="glr_prefill", op="glr", dir="fwd", dtype="bf16", batch=1, seqlen=32749, dim=1536, resets=False),
        # Training with packed documents, float32 storage.
        dict(name="glr_train_f32", op="glr", dir="train", dtype="f32", batch=8, seqlen=2048, dim=1536, resets=True),
        # Training at the width and length of the large-channel scan.
        dict(name="glr_train", op="glr", dir="train", dtype="bf16", batch=4, seqlen=4096, dim=5120, resets=True),
        # Norm before a mixer while decoding 32 sequences: the smallest call.
        dict(name="rms_step", op="rms", dir="fwd", dtype="bf16", rows=32, dim=1024, group=0),
        # Prefill that feeds an 8-bit product, one scale per token.
        dict(name="rms_q8", op="rms", dir="q8", dtype="bf16", rows=16384, dim=5120, group=0),
        # Training, the ordinary width.
        dict(name="rms_train", op="rms", dir="train", dtype="bf16", rows=16384, dim=2048, group=0),
        # Odd rows and an odd width: rows start at no vector boundary.
        dict(name="rms_train_odd", op="rms", dir="train", dtype="f32", rows=4095, dim=1537, group=0),
        # Prefill of one long prompt, 16 query heads on 4 key heads.
        dict(name="swa_prefill", op="swa", dir="fwd", dtype="bf16", batch=1, seqlen=8192, heads=16, kv_heads=4,
             headdim=128, window=1024, sinks=4, ragged=False),
        # Training on rows of unequal length, 32 heads of 64.
        dict(name="swa_train", op="swa", dir="train", dtype="bf16", batch=4, seqlen=2048, heads=32, kv_heads=8,
             headdim=64, window=512, sinks=4, ragged=True),
        # One token of 4 sequences: latency.
        dict(name="swa_step", op="swa", dir="step", dtype="bf16", batch=4, seqlen=1, heads=16, kv_heads=4,
             headdim=128, window=1024, sinks=4, ragged=False),
        # One token of 64 sequences over long windows: the cache is read once.
        dict(name="swa_step_64", op="swa", dir="step", dtype="bf16", batch=64, seqlen=1, heads=32, kv_heads=8,
             headdim=128, window=4096, sinks=4, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, way = rng.choice([("glr", "step"), ("glr", "fwd"), ("glr", "train"), ("rms", "fwd"), ("rms", "q8"),
                          ("rms", "train"), ("swa", "fwd"), ("swa", "train"), ("swa", "step")])
    if op == "glr":
        dim = _log_int(rng, 256, 5120)
        if rng.random() < 0.5:
            dim = max(64, dim // 64 * 64)
        batch = _log_int(rng, 1, 128 if way == "step" else 8)
        most = 4 * 4096 * 5120 // (batch * dim)
        seqlen = 1 if way == "step" else _log_int(rng, 64, min(32768, most))
        return dict(op=op, dir=way, dtype=rng.choice(["bf16", "bf16", "f32"]), batch=batch, seqlen=seqlen, dim=dim,
                    resets=rng.random() < 0.5 and way != "step")
    if op == "rms":
        dim = _log_int(rng, 128, 8192)
        if rng.random() < 0.5:
            dim = dim // 64 * 64
        rows = _log_int(rng, 1, min(32768, 16384 * 5120 // dim))
        return dict(op=op, dir=way, dtype=rng.choice(["bf16", "bf16", "f32"]), rows=rows, dim=dim,
                    group=rng.choice([0, 128]) if way == "q8" else 0)
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 8] if kv_heads < 8 else [1, 2, 4])
    case = dict(op=op, dir=way, dtype="bf16", heads=heads, kv_heads=kv_heads, headdim=rng.choice([64, 128]),
                window=_log_int(rng, 64, 4096), sinks=rng.choice([0, 1, 4, 16]), ragged=rng.random() < 0.5)
    if way == "step":
        return dict(case, batch=_log_int(rng, 1, 64), seqlen=1)
    case["window"] = min(case["window"], 1024)
    case["batch"] = _log_int(rng, 1, 4)
    most = 4 * 32 * 2048 ** 2 // (1 if way == "train" else 2)
    case["seqlen"] = _log_int(rng, 128, min(8192, math.isqrt(most // (case["batch"] * heads))))
    return case


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)

    st = dict(case)
    if case["op"] == "glr":
        b, n, d = case["batch"], case["seqlen"], case["dim"]
        # Decay rates from slow (a = 0.996 at an open gate) to fast (a = 0.02).
        st["A"] = -torch.exp(math.log(0.004) + uniform(d) * math.log(4.0 / 0.004))
        st["h0"] = normal(b, d, dtype=torch.float32)
        lead = (b, d) if case["dir"] == "step" else (b, n, d)
        for k in ("x", "rec", "inp"):
            st[k] = normal(*lead)
        st["reset"] = (uniform(b, n) < 1 / 256).to(torch.uint8) if case["resets"] else None
        if case["dir"] == "train":
            st["dy"] = normal(b, n, d)
    elif case["op"] == "rms":
        rows, d = case["rows"], case["dim"]
        st["x"], st["residual"] = normal(rows, d), normal(rows, d, std=2.0)
        st["w"] = 1.0 + 0.1 * normal(d, dtype=torch.float32)
        if case["dir"] == "train":
            st["dy"], st["dres"] = normal(rows, d), normal(rows, d)
    else:
        b, n, h, kv, d = case["batch"], case["seqlen"], case["heads"], case["kv_heads"], case["headdim"]
        # One fused projection holds queries, keys and values side by side.
        qkv = normal(b, n, (h + 2 * kv) * d)
        st["q"] = qkv[..., :h * d].view(b, n, h, d)
        st["k"] = qkv[..., h * d:(h + kv) * d].view(b, n, kv, d)
        st["v"] = qkv[..., (h + kv) * d:].view(b, n, kv, d)
        if case["dir"] == "step":
            slots = case["window"] + case["sinks"]
            st["k_cache"], st["v_cache"] = normal(b, kv, slots, d), normal(b, kv, slots, d)
            # Sequences that have run past the window, or (ragged) are anywhere up to twice it.
            at = uniform(b) * 2 * slots if case["ragged"] else slots + uniform(b) * slots
            st["pos"] = at.to(torch.int32)
        else:
            st["lengths"] = None
            if case["ragged"]:
                st["lengths"] = (n * (0.25 + 0.75 * uniform(b))).ceil().to(torch.int32)
            if case["dir"] == "train":
                st["dy"] = normal(b, n, h, d)
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1, by doubling the span each step covers."""
    k = 1
    while k < a.shape[1]:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _plain_glr(st):
    step, train = st["dir"] == "step", st["dir"] == "train"
    up = (lambda t: t.float()[:, None]) if step else (lambda t: t.float())
    x, r, i, A = up(st["x"]), torch.sigmoid(up(st["rec"])), torch.sigmoid(up(st["inp"])), st["A"]
    a = torch.exp(A * r)
    beta = torch.sqrt(-torch.expm1(2 * A * r))
    carry = a if st["reset"] is None else a * (st["reset"] == 0)[..., None]
    b = beta * i * x
    b[:, 0] += carry[:, 0] * st["h0"]
    h = _scan(carry, b)
    y = h.to(st["x"].dtype)
    h_last = h[:, -1].clone()
    if not train:
        return (y[:, 0], h_last) if step else (y, h_last)
    after = torch.cat([carry[:, 1:], torch.zeros_like(carry[:, :1])], 1)
    g = _scan(after.flip(1), st["dy"].float().flip(1)).flip(1)
    from_prev = carry * torch.cat([st["h0"][:, None], h[:, :-1]], 1)
    slope = torch.where(beta > 0, a * a / beta, torch.zeros_like(a))
    dla = g * (from_prev - slope * i * x)
    out = (g * beta * i, dla * A * r * (1 - r), g * beta * x * i * (1 - i))
    return (y, h_last) + tuple(t.to(y.dtype) for t in out) + ((dla * r).sum((0, 1)), carry[:, 0] * g[:, 0])


def _plain_rms(st):
    s = st["x"].float() + st["residual"].float()
    rstd = torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS)
    n = s * rstd
    y, dt = n * st["w"], st["x"].dtype
    if st["dir"] == "fwd":
        return y.to(dt), s.to(dt)
    if st["dir"] == "q8":
        group = st["group"] or y.shape[1]
        pad = -y.shape[1] % group
        wide = torch.nn.functional.pad(y, (0, pad)).view(y.shape[0], -1, group)
        scale = wide.abs().amax(-1) / 448.0
        q = (wide / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]).clamp(-448.0, 448.0)
        return q.reshape(y.shape[0], -1)[:, :y.shape[1]].to(torch.float8_e4m3fn), scale, s.to(dt)
    # The backward of a training step reads the sum as it was stored.
    kept = s.to(dt).float()
    rstd = torch.rsqrt((kept * kept).mean(-1, keepdim=True) + EPS)
    n = kept * rstd
    dy = st["dy"].float()
    dn = dy * st["w"]
    dx = rstd * (dn - n * (dn * n).mean(-1, keepdim=True)) + st["dres"].float()
    return y.to(dt), s.to(dt), dx.to(dt), (dy * n).sum(0)


def _plain_swa(st):
    if st["dir"] == "step":
        return _plain_swa_step(st)
    q, k, v = (st[t].float().transpose(1, 2) for t in ("q", "k", "v"))
    b, h, n, d = q.shape
    kv = k.shape[1]
    q = q.reshape(b, kv, h // kv, n, d)
    k, v = k[:, :, None], v[:, :, None]
    t = torch.arange(n, device=q.device)
    gap = t[:, None] - t[None, :]
    sees = (gap >= 0) & ((gap < st["window"]) | (t[None, :] < st["sinks"]))
    if st["lengths"] is not None:
        within = t < st["lengths"][:, None]
        sees = (sees & within[:, :, None] & within[:, None, :])[:, None, None]
    scale = 1 / math.sqrt(d)
    s = (q @ k.transpose(-1, -2) * scale).masked_fill(~sees, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    del s
    o = p @ v
    dt = st["q"].dtype

    def heads_last(t):
        return t.reshape(b, -1, n, d).transpose(1, 2).to(dt)

    y = heads_last(o)
    if st["dir"] == "fwd":
        return y
    do = st["dy"].float().transpose(1, 2).reshape(b, kv, h // kv, n, d)
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
    dq = ds @ k * scale
    dk = (ds.transpose(-1, -2) @ q * scale).sum(2)
    return y, heads_last(dq), heads_last(dk), heads_last(dv)


def _plain_swa_step(st):
    pos, sinks, window = st["pos"].long(), st["sinks"], st["window"]
    rows = torch.arange(pos.shape[0], device=pos.device)
    slot = torch.where(pos < sinks, pos, sinks + (pos - sinks) % window)
    st["k_cache"][rows, :, slot] = st["k"][:, 0]
    st["v_cache"][rows, :, slot] = st["v"][:, 0]
    k, v = st["k_cache"].float(), st["v_cache"].float()
    b, kv, slots, d = k.shape
    q = st["q"].float().view(b, kv, -1, d)
    s = q @ k.transpose(-1, -2) / math.sqrt(d)
    s = s.masked_fill((torch.arange(slots, device=pos.device) > pos[:, None])[:, None, None], -math.inf)
    p = torch.softmax(s, -1)
    return (p @ v).view(b, -1, d).to(st["q"].dtype), st["k_cache"], st["v_cache"]


# ---------------------------------------------------------------------------
# The library's entry points
# ---------------------------------------------------------------------------

def _own_glr(st):
    import state_space_model_ssm_amd as ssm
    if st["dir"] == "step":
        return ssm.glr_step(st["x"], st["rec"], st["inp"], st["A"], st["h0"], h_out=torch.empty_like(st["h0"]))
    args = (st["x"], st["rec"], st["inp"], st["A"])
    if st["dir"] == "fwd":
        return ssm.glr_fwd(*args, h0=st["h0"], reset=st["reset"])
    y, h_last, states = ssm.glr_fwd(*args, h0=st["h0"], reset=st["reset"], return_states=True)
    return (y, h_last) + tuple(ssm.glr_bwd(*args, states, st["dy"], reset=st["reset"]))


def _own_rms(st):
    import state_space_model_ssm_amd as ssm
    if st["dir"] == "q8":
        return ssm.rms_add_q8_fwd(st["x"], st["w"], st["residual"], eps=EPS, group=st["group"])
    y, s = ssm.rms_add_fwd(st["x"], st["w"], st["residual"], eps=EPS)
    if st["dir"] == "fwd":
        return y, s
    return (y, s) + tuple(ssm.rms_add_bwd(st["dy"], s, st["w"], dres=st["dres"], eps=EPS))


def _own_swa(st):
    import state_space_model_ssm_amd as ssm
    if st["dir"] == "step":
        y = ssm.swa_step(st["q"][:, 0], st["k"][:, 0], st["v"][:, 0], st["k_cache"], st["v_cache"], st["pos"],
                         sinks=st["sinks"])
        return y, st["k_cache"], st["v_cache"]
    args, kw = (st["q"], st["k"], st["v"]), dict(window=st["window"], sinks=st["sinks"], lengths=st["lengths"])
    y, lse = ssm.swa_fwd(*args, **kw)
    if st["dir"] == "fwd":
        return y
    return (y,) + tuple(ssm.swa_bwd(*args, y, lse, st["dy"], **kw))


def run(st):
    plain, kernels = {"glr": (_plain_glr, _own_glr), "rms": (_plain_rms, _own_rms),
                      "swa": (_plain_swa, _own_swa)}[st["op"]]
    return kernels(st) if own else plain(st)


# ---------------------------------------------------------------------------
# Bytes and operations
# ---------------------------------------------------------------------------

def _pairs(case):
    """Query-key pairs of one head over the batch, at full lengths (or their mean, 5/8, where they are ragged)."""
    n = case["seqlen"] * (0.625 if case["ragged"] else 1.0)
    w = min(case["window"], n)
    return case["batch"] * (n * w - w * (w - 1) / 2 + max(0.0, n - w) * min(case["sinks"], n))


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    train = case["dir"] == "train"
    if case["op"] == "glr":
        n = case["batch"] * case["seqlen"] * case["dim"]
        ends = 4 * case["batch"] * case["dim"]
        return {"bytes": n * e * (8 if train else 4) + ends * 2, "flops": n * (60 if train else 20)}
    if case["op"] == "rms":
        n = case["rows"] * case["dim"]
        if case["dir"] == "q8":
            return {"bytes": n * (3 * e + 1), "flops": 8 * n}
        return {"bytes": n * e * (7 if train else 4), "flops": n * (20 if train else 6)}
    b, h, kv, d = case["batch"], case["heads"], case["kv_heads"], case["headdim"]
    if case["dir"] == "step":
        slots = case["window"] + case["sinks"]
        keys = b * slots * (0.75 if case["ragged"] else 1.0)
        return {"bytes": 2 * e * d * (keys * kv + b * (h + kv)), "flops": 4 * d * h * keys}
    rows = b * case["seqlen"]
    size = rows * d * e
    pairs = _pairs(case)
    if train:
        return {"bytes": size * (4 * h + 4 * kv - h), "flops": 14 * d * h * pairs}
    return {"bytes": size * (2 * h + 2 * kv), "flops": 4 * d * h * pairs}


# ---------------------------------------------------------------------------
# The definitions in float64
# ---------------------------------------------------------------------------

def _exact_glr(st):
    train, step = st["dir"] == "train", st["dir"] == "step"
    x, rec, inp = (st[k].double().unsqueeze(1) if step else st[k].double() for k in ("x", "rec", "inp"))
    A, n = st["A"].double(), x.shape[1]
    r, i = 1 / (1 + torch.exp(-rec)), 1 / (1 + torch.exp(-inp))
    a = torch.exp(A * r)
    b = torch.sqrt((1 - a) * (1 + a))
    keep = torch.ones(x.shape[:2], dtype=torch.float64, device=x.device)
    if st["reset"] is not None:
        keep = 1 - st["reset"].double()
    u, ka = b * i * x, a * keep[..., None]
    h = torch.empty_like(x)
    prev = st["h0"].double()
    for t in range(n):
        prev = torch.addcmul(u[:, t], ka[:, t], prev, out=h[:, t])
    if not train:
        return (h[:, 0], h[:, -1]) if step else (h, h[:, -1])
    g = st["dy"].double()
    for t in range(n - 2, -1, -1):
        g[:, t] += ka[:, t + 1] * g[:, t + 1]
    before = torch.cat([st["h0"].double()[:, None], h[:, :-1]], 1)
    # d h / d log a, holding h_{t-1}: a h_{t-1} from the decay, -a^2 / b i x from the input's weight.
    log_a = g * (ka * before - a * a / b * i * x)
    dx, drec, dinp = g * b * i, log_a * A * r * (1 - r), g * b * x * i * (1 - i)
    return h, h[:, -1], dx, drec, dinp, (log_a * r).sum((0, 1)), ka[:, 0] * g[:, 0]


def _exact_rms(st):
    s = st["x"].double() + st["residual"].double()
    norm = s / (s.pow(2).sum(-1, keepdim=True) / s.shape[1] + EPS).sqrt()
    y = norm * st["w"].double()
    if st["dir"] == "fwd":
        return y, s
    if st["dir"] == "q8":
        group = st["group"] or y.shape[1]
        parts = [t.abs().max(1).values / 448 for t in y.split(group, 1)]
        return torch.cat([t / c[:, None] for t, c in zip(y.split(group, 1), parts)], 1), torch.stack(parts, 1), s
    z = s.to(st["x"].dtype).double().requires_grad_(True)
    w = st["w"].double().requires_grad_(True)
    out = z / (z.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w
    dz, dw = torch.autograd.grad(out, (z, w), st["dy"].double())
    return y, s, dz + st["dres"].double(), dw


def _exact_swa(st):
    step = st["dir"] == "step"
    train = st["dir"] == "train"
    q = st["q"].double()
    b, n, heads, d = q.shape
    group = heads // st["kv_heads"]
    if step:
        keys, values = st["k_cache"].clone(), st["v_cache"].clone()
        y = torch.zeros(b, heads, d, dtype=torch.float64, device=q.device)
        for row in range(b):
            p = int(st["pos"][row])
            slot = p if p < st["sinks"] else st["sinks"] + (p - st["sinks"]) % st["window"]
            keys[row, :, slot], values[row, :, slot] = st["k"][row, 0], st["v"][row, 0]
            count = min(p + 1, keys.shape[2])
            for c in range(st["kv_heads"]):
                e = torch.exp(q[row, 0, c * group:(c + 1) * group] @ keys[row, c, :count].double().T / math.sqrt(d))
                y[row, c * group:(c + 1) * group] = e @ values[row, c, :count].double() / e.sum(1, keepdim=True)
        return y, keys.double(), values.double()
    y, dq = torch.zeros_like(q), torch.zeros_like(q)
    dk = torch.zeros(b, n, st["kv_heads"], d, dtype=torch.float64, device=q.device)
    dv = torch.zeros_like(dk)
    for row in range(b):
        m = n if st["lengths"] is None else int(st["lengths"][row])
        at = torch.arange(m, device=q.device)
        hidden = at[None] > at[:, None]
        hidden |= (at[:, None] - at[None] >= st["window"]) & (at[None] >= st["sinks"])
        for head in range(heads):
            c = head // group
            qh, kh, vh = q[row, :m, head], st["k"][row, :m, c].double(), st["v"][row, :m, c].double()
            e = torch.exp(qh @ kh.T / math.sqrt(d)).masked_fill(hidden, 0.0)
            p = e / e.sum(1, keepdim=True)
            y[row, :m, head] = p @ vh
            if train:
                do = st["dy"][row, :m, head].double()
                dp = do @ vh.T
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(d)
                dq[row, :m, head] = ds @ kh
                dk[row, :m, c] += ds.T @ qh
                dv[row, :m, c] += p.T @ do
    return (y, dq, dk, dv) if train else y


def exact(case, seed):
    return {"glr": _exact_glr, "rms": _exact_rms, "swa": _exact_swa}[case["op"]](prepare(case, seed))
