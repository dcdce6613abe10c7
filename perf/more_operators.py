"""Work of the operators of delta-rule and normalised-attention blocks: the
gated delta rule, norms of queries and keys with the position rotation, and
attention steps over a cache held in 8 bits.

Every case is one call (or, for "train", the forward with its backward) on
data that a model's program holds at that point.  ``run`` computes it with
elementary torch operations in float32, or through the library's entry points
when ``own`` is set; ``exact`` computes it from the definitions in float64.

Definitions:
  gdr   per value head, with a_t = exp(g_t) and the state S (V x K):
        u_t = beta_t (v_t - a_t S_{t-1} k_t),  S_t = a_t S_{t-1} + u_t k_t',
        y_t = scale S_t q_t;  query and key heads may be shared by value heads
  qkn   per head of q and of k: n = x / sqrt(mean(x^2) + eps) * w, then its
        first 2 len(inv_freq) elements are rotated in pairs by pos * inv_freq
  swa8  one token against a cache of the last `window` positions in e4m3
        floats with one float32 scale per block of 64 positions and head; the
        sinks and the block that is being filled are bfloat16, and a block is
        stored in 8 bits, scale amax / 448, when its last position comes
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
BLOCK = 64


def listed():
    return [
        # One token of 4 sequences through a delta-rule layer: latency.
        dict(name="gdr_step", op="gdr", dir="step", dtype="bf16", gates="f32", batch=4, seqlen=1, qk_heads=16, heads=16,
             kdim=128, vdim=128, ragged=False, state=True),
        # One token of 64 sequences, 32 value heads on 16: the states are read and written once.
        dict(name="gdr_step_64", op="gdr", dir="step", dtype="bf16", gates="f32", batch=64, seqlen=1, qk_heads=16,
             heads=32, kdim=128, vdim=128, ragged=False, state=True),
        # One long prompt: few heads, so time itself has to be shared out.
        dict(name="gdr_prefill", op="gdr", dir="fwd", dtype="bf16", gates="f32", batch=1, seqlen=8192, qk_heads=16,
             heads=16, kdim=128, vdim=128, ragged=False, state=False),
        # The next piece of several prompts of unequal, odd lengths, from a state; heads of 64.
        dict(name="gdr_prefill_odd", op="gdr", dir="fwd", dtype="bf16", gates="bf16", batch=3, seqlen=1999, qk_heads=8,
             heads=32, kdim=64, vdim=64, ragged=True, state=True),
        # Training, heads of 128.
        dict(name="gdr_train", op="gdr", dir="train", dtype="bf16", gates="bf16", batch=4, seqlen=2048, qk_heads=16,
             heads=16, kdim=128, vdim=128, ragged=False, state=False),
        # Training on rows of unequal length, keys of 64 shared by two value heads of 128.
        dict(name="gdr_train_shared", op="gdr", dir="train", dtype="bf16", gates="bf16", batch=2, seqlen=1021,
             qk_heads=8, heads=16, kdim=64, vdim=128, ragged=True, state=False),
        # Queries and keys of one token of 32 sequences: the smallest call.
        dict(name="qkn_step", op="qkn", dir="fwd", dtype="bf16", batch=32, seqlen=1, heads=16, kv_heads=4, headdim=128,
             rot=128, far=True, pairs="halves"),
        # One long prompt of odd length at positions far from the start.
        dict(name="qkn_prefill", op="qkn", dir="fwd", dtype="bf16", batch=1, seqlen=32749, heads=16, kv_heads=4,
             headdim=128, rot=128, far=True, pairs="halves"),
        # Training, heads of 64, half of each rotated.
        dict(name="qkn_train", op="qkn", dir="train", dtype="bf16", batch=4, seqlen=2048, heads=32, kv_heads=8,
             headdim=64, rot=32, far=False, pairs="neighbours"),
        # One token of 4 sequences against windows in 8 bits: latency.
        dict(name="swa8_step", op="swa8", dir="step", dtype="bf16", batch=4, heads=16, kv_heads=4, headdim=128,
             window=1024, sinks=4, ragged=False),
        # One token of 64 sequences over long windows: the cache is read once.
        dict(name="swa8_step_64", op="swa8", dir="step", dtype="bf16", batch=64, heads=32, kv_heads=8, headdim=128,
             window=4096, sinks=4, ragged=True),
        # Prompts of unequal length into 8-bit caches.
        dict(name="swa8_fill", op="swa8", dir="fill", dtype="bf16", batch=8, seqlen=8192, heads=32, kv_heads=8,
             headdim=128, window=4096, sinks=4, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op, way = rng.choice([("gdr", "step"), ("gdr", "fwd"), ("gdr", "fwd"), ("gdr", "train"), ("gdr", "train"),
                          ("qkn", "fwd"), ("qkn", "train"), ("swa8", "step"), ("swa8", "step"), ("swa8", "fill")])
    if op == "gdr":
        kdim, vdim = rng.choice([64, 128]), rng.choice([64, 128])
        qk_heads = rng.choice([1, 2, 4, 8, 16])
        heads = qk_heads * rng.choice([1, 2, 4] if qk_heads < 16 else [1, 2])
        case = dict(op=op, dir=way, dtype="bf16", gates="bf16" if way == "train" else rng.choice(["bf16", "f32"]),
                    qk_heads=qk_heads, heads=heads, kdim=kdim, vdim=vdim)
        if way == "step":
            return dict(case, batch=_log_int(rng, 1, 64), seqlen=1, ragged=False, state=True)
        case["batch"] = _log_int(rng, 1, 8)
        most = 8192 * 16 * 128 * 128 // (case["batch"] * heads * kdim * vdim)
        case["seqlen"] = _log_int(rng, 16, min(8192, most))
        return dict(case, ragged=rng.random() < 0.5, state=rng.random() < 0.5 and way == "fwd")
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 8] if kv_heads < 8 else [1, 2, 4])
    case = dict(op=op, dir=way, dtype="bf16", heads=heads, kv_heads=kv_heads)
    if op == "qkn":
        headdim = rng.choice([64, 96, 128, 256])
        rot = rng.choice([r for r in (32, 64, 96, 128, 256) if r <= headdim])
        batch = _log_int(rng, 1, 64)
        most = 32749 * 20 * 128 // (batch * (heads + kv_heads) * headdim * (2 if way == "train" else 1))
        return dict(case, dtype=rng.choice(["bf16", "bf16", "f32"]), batch=batch,
                    seqlen=_log_int(rng, 1, min(32768, max(1, most))), headdim=headdim, rot=rot,
                    far=rng.random() < 0.5, pairs=rng.choice(["halves", "neighbours"]))
    case.update(headdim=rng.choice([64, 128]), window=BLOCK * _log_int(rng, 1, 64), sinks=rng.choice([0, 1, 4, 16]),
                ragged=rng.random() < 0.5)
    if way == "step":
        return dict(case, batch=_log_int(rng, 1, 64))
    batch = _log_int(rng, 1, 8)
    return dict(case, batch=batch, seqlen=_log_int(rng, 16, 8192))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)

    st = dict(case)
    b, n = case["batch"], case.get("seqlen", 1)
    if case["op"] == "gdr":
        h, qk, kd, vd = case["heads"], case["qk_heads"], case["kdim"], case["vdim"]
        # Keys and queries of unit length, as their norm before the rule makes them.
        st["q"], st["k"] = (torch.nn.functional.normalize(normal(b, n, qk, kd, dtype=torch.float32), dim=-1).to(dt)
                            for _ in range(2))
        st["v"] = normal(b, n, h, vd)
        # Heads from slow (a = 0.999 a step) to fast (a = 0.4), and gates around the middle.
        rate = torch.exp(math.log(0.001) + uniform(h) * math.log(1.0 / 0.001))
        gates = DTYPES[case["gates"]]
        st["g"] = (-rate * torch.nn.functional.softplus(normal(b, n, h, dtype=torch.float32))).to(gates)
        st["beta"] = torch.sigmoid(normal(b, n, h, dtype=torch.float32)).to(gates)
        st["h0"] = normal(b, h, vd, kd, dtype=torch.float32, std=0.5) if case["state"] else None
        st["lengths"] = (n * (0.25 + 0.75 * uniform(b))).ceil().to(torch.int32) if case["ragged"] else None
        if case["dir"] == "step":
            for t in ("q", "k", "v", "g", "beta"):
                st[t] = st[t][:, 0].contiguous()
            st["h_out"] = torch.empty_like(st["h0"])
        elif case["dir"] == "train":
            st["dy"] = normal(b, n, h, vd)
        return st
    h, kv, d = case["heads"], case["kv_heads"], case["headdim"]
    # One fused projection holds queries, keys and values side by side.
    qkv = normal(b, n, (h + 2 * kv) * d)
    st["q"] = qkv[..., :h * d].view(b, n, h, d)
    st["k"] = qkv[..., h * d:(h + kv) * d].view(b, n, kv, d)
    st["v"] = qkv[..., (h + kv) * d:].view(b, n, kv, d)
    if case["op"] == "qkn":
        st["wq"], st["wk"] = (1.0 + 0.1 * normal(d, dtype=torch.float32) for _ in range(2))
        half = case["rot"] // 2
        st["inv_freq"] = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        start = (uniform(b, 1) * (1 << 20) if case["far"] else uniform(b, 1) * 0).to(torch.int32)
        st["pos"] = start + torch.arange(n, device="cuda", dtype=torch.int32)
        if case["dir"] == "train":
            st["dq"], st["dk"] = normal(b, n, h, d), normal(b, n, kv, d)
        return st
    window, sinks = case["window"], case["sinks"]
    st["cache"] = [normal(b, kv, sinks + BLOCK, d) for _ in range(2)]
    st["cache"] += [normal(b, kv, window, d, std=100.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn) for _ in range(2)]
    st["cache"] += [(0.5 + uniform(b, kv, window // BLOCK)) / 100 for _ in range(2)]
    if case["dir"] == "fill":
        st["lengths"] = (n * (0.25 + 0.75 * uniform(b))).ceil().to(torch.int32) if case["ragged"] else None
        return st
    # Sequences that have run past the window, or (ragged) are anywhere up to twice it; the first one's block fills up.
    at = (uniform(b) * 2 * window if case["ragged"] else (1 + uniform(b)) * window).to(torch.int32)
    at[0] = at[0] // BLOCK * BLOCK + BLOCK - 1
    st["pos"] = at + sinks
    for t in ("q", "k", "v"):
        st[t] = st[t][:, 0]
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _chunks(t, n):
    """(b, L, h, ...) -> (b, h, chunks, n, ...), zeros behind the end."""
    t = t.transpose(1, 2)
    pad = -t.shape[2] % n
    if pad:
        t = torch.cat([t, t.new_zeros(*t.shape[:2], pad, *t.shape[3:])], 2)
    return t.unflatten(2, (-1, n))


def _delta_rule(q, k, v, g, beta, h0, lengths, scale):
    """(y, state after the last token): chunks of 64 tokens, products within them, the state from one to the next."""
    b, n, h, vd = v.shape
    share = h // q.shape[2]
    if lengths is not None:
        within = (torch.arange(n, device=v.device) < lengths[:, None])[..., None]
        g, beta = g.masked_fill(~within, 0.0), beta.masked_fill(~within, 0.0)
    q, k, v, g, beta = (_chunks(t, BLOCK) for t in (q, k, v, g, beta))
    q, k = (t.repeat_interleave(share, 1) if share > 1 else t for t in (q, k))
    sums = g.double().cumsum(-1)
    i = torch.arange(BLOCK, device=v.device)
    gap = (sums[..., :, None] - sums[..., None, :]).masked_fill(i[:, None] < i, -math.inf)
    decay = torch.exp(gap).float()
    kk = (k @ k.transpose(-1, -2)) * decay * (i[:, None] > i)
    eye = torch.eye(BLOCK, device=v.device)
    # (I + low)^-1 = (I - low)(I + low^2)(I + low^4)...: low^64 = 0.
    low = beta[..., None] * kk
    inv, power = eye - low, low @ low
    for _ in range(5):
        inv, power = inv @ (eye + power), power @ power
    att = (q @ k.transpose(-1, -2)) * decay * scale
    into, last = torch.exp(sums).float()[..., None], sums[..., -1:]
    out = torch.exp(last - sums).float()[..., None]
    u0, w = inv @ (beta[..., None] * v), inv @ (beta[..., None] * into * k)
    kout, whole = (out * k).transpose(-1, -2), torch.exp(last).float()[..., None]
    s = k.new_zeros(b, h, k.shape[-1], vd) if h0 is None else h0.transpose(-1, -2)
    before, us = [], []
    for c in range(k.shape[2]):
        before.append(s)
        us.append(u0[:, :, c] - w[:, :, c] @ s)
        s = whole[:, :, c] * s + kout[:, :, c] @ us[-1]
    y = (scale * into * q) @ torch.stack(before, 2) + att @ torch.stack(us, 2)
    y = y.flatten(2, 3)[:, :, :n].transpose(1, 2)
    if lengths is not None:
        y = y * within[..., None]
    return y, s.transpose(-1, -2)


def _plain_gdr(st):
    names = ("q", "k", "v", "g", "beta")
    scale = st["kdim"] ** -0.5
    if st["dir"] == "step":
        q, k, v, g, beta = (st[t].float() for t in names)
        share = v.shape[1] // q.shape[1]
        q, k = q.repeat_interleave(share, 1), k.repeat_interleave(share, 1)
        s = st["h0"] * torch.exp(g)[..., None, None]
        u = beta[..., None] * (v - (s * k[:, :, None]).sum(-1))
        s = s + u[..., None] * k[:, :, None]
        return ((s * q[:, :, None]).sum(-1) * scale).to(st["v"].dtype), s
    x = [st[t].float() for t in names]
    train = st["dir"] == "train"
    if train:
        x = [t.requires_grad_(True) if t.is_leaf and t is not st[n] else t.clone().requires_grad_(True)
             for t, n in zip(x, names)]
    y, s = _delta_rule(*x, st["h0"], st["lengths"], scale)
    if not train:
        return y.to(st["v"].dtype), s
    grads = torch.autograd.grad(y, x, st["dy"].float())
    return (y.detach().to(st["v"].dtype),) + tuple(t.to(st[n].dtype) for t, n in zip(grads, names))


def _turn(x, cos, sin, pairs):
    """x's first elements rotated in pairs; cos, sin: (..., 1, half)."""
    half = cos.shape[-1]
    if pairs == "halves":
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_qkn(st):
    angle = (st["pos"].double()[..., None] * st["inv_freq"].double())[..., None, :]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    outs, grads = [], []
    for name, w in (("q", st["wq"]), ("k", st["wk"])):
        x = st[name].float()
        rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        n = x * rstd
        outs.append(_turn(n * w, cos, sin, st["pairs"]).to(st[name].dtype))
        if st["dir"] == "train":
            dn = _turn(st["d" + name].float(), cos, -sin, st["pairs"])
            dw = (dn * n).sum((0, 1, 2))
            dn = dn * w
            grads += [(rstd * (dn - n * (dn * n).mean(-1, keepdim=True))).to(st[name].dtype), dw]
    return tuple(outs + grads)


def _quantise(blocks):
    """(..., block, d) float32 -> e4m3 values and a scale per block."""
    scale = blocks.abs().amax((-1, -2)) / 448.0
    per = torch.where(scale > 0, scale, torch.ones_like(scale))[..., None, None]
    return (blocks / per).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _plain_swa8_fill(st):
    """Whatever a next token would see of the prompts: sinks and the last block's tokens as they are, whole blocks in 8 bits."""
    window, sinks = st["window"], st["sinks"]
    b, n, kv, d = st["k"].shape
    length = torch.full((b,), n, device="cuda") if st["lengths"] is None else st["lengths"].long()
    ring = torch.arange(window // BLOCK, device="cuda")
    count = (length - sinks).clamp_min(0)
    done = count // BLOCK                                        # blocks that are whole
    last = (done[:, None] - 1 - ring) // ring.shape[0] * ring.shape[0] + ring
    has = (done[:, None] > ring) & (last >= 0)
    where = (sinks + last.clamp_min(0)[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")).clamp_max(n - 1)
    slot = torch.arange(sinks + BLOCK, device="cuda").expand(b, -1)
    tail = torch.where(slot < sinks, slot, slot + (done * BLOCK)[:, None])
    held = tail < length[:, None]
    rows = torch.arange(b, device="cuda")[:, None]
    for k, t in enumerate(("k", "v")):
        near, ring8, scale = st["cache"][k], st["cache"][2 + k], st["cache"][4 + k]
        near.copy_(torch.where(held[:, None, :, None], st[t][rows, tail.clamp_max(n - 1)].transpose(1, 2), near))
        blocks = st[t][rows[..., None], where].permute(0, 3, 1, 2, 4).float()
        q, s = _quantise(blocks)
        scale.copy_(torch.where(has[:, None], s, scale))
        keep = has[:, None, :, None, None]
        bits = torch.where(keep, q.view(torch.uint8), ring8.view(torch.uint8).view(b, kv, -1, BLOCK, d))
        ring8.view(torch.uint8).copy_(bits.view(b, kv, window, d))
    return tuple(st["cache"])


def _plain_swa8(st):
    if st["dir"] == "fill":
        return _plain_swa8_fill(st)
    window, sinks, pos = st["window"], st["sinks"], st["pos"].long()
    b, kv = st["k"].shape[:2]
    d = st["k"].shape[-1]
    rows = torch.arange(b, device="cuda")
    spot = (pos - sinks).clamp_min(0)
    place, block = spot % BLOCK, spot % window // BLOCK
    slot = torch.where(pos < sinks, pos, sinks + place)
    for k, t in enumerate(("k", "v")):
        st["cache"][k][rows, :, slot] = st[t]
    # Positions that the ring holds: those of whole blocks, except the block being filled up to the token.
    at = torch.arange(window, device="cuda")
    in_block = at // BLOCK == block[:, None]
    ring_ok = torch.where(in_block, at % BLOCK > place[:, None], True) & (pos[:, None] >= sinks)
    ring_ok &= torch.where(at > (spot % window)[:, None], spot[:, None] >= window, True)
    near = torch.arange(sinks + BLOCK, device="cuda")
    near_ok = torch.where(near < sinks, near <= pos[:, None], (near - sinks <= place[:, None]) & (pos[:, None] >= sinks))
    values = []
    for k in range(2):
        wide = st["cache"][2 + k].float().view(b, kv, -1, BLOCK, d) * st["cache"][4 + k][..., None, None]
        values.append(torch.cat([st["cache"][k].float(), wide.view(b, kv, window, d)], 2))
    ok = torch.cat([near_ok, ring_ok], 1)[:, None, None]    # (b, 1, 1, places)
    s = st["q"].float().reshape(b, kv, -1, d) @ values[0].transpose(-1, -2) / math.sqrt(d)
    s = s.masked_fill(~ok, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    y = (p @ values[1].masked_fill(~ok.transpose(-1, -2), 0.0)) / p.sum(-1, keepdim=True)
    full = ((place == BLOCK - 1) & (pos >= sinks))[:, None]
    for k in range(2):
        q, scale = _quantise(st["cache"][k][:, :, sinks:].float())
        st["cache"][4 + k][rows, :, block] = torch.where(full, scale, st["cache"][4 + k][rows, :, block])
        ring8 = st["cache"][2 + k].view(torch.uint8).view(b, kv, -1, BLOCK, d)
        ring8[rows, :, block] = torch.where(full[..., None, None], q.view(torch.uint8), ring8[rows, :, block])
    return (y.reshape(b, -1, d).to(st["q"].dtype), *st["cache"])


# ---------------------------------------------------------------------------
# The library's entry points
# ---------------------------------------------------------------------------

def _own_gdr(st):
    import state_space_model_ssm_amd as ssm
    args = tuple(st[t] for t in ("q", "k", "v", "g", "beta"))
    if st["dir"] == "step":
        return ssm.gdr_step(*args, st["h0"], h_out=st["h_out"])
    if st["dir"] == "fwd":
        return ssm.gdr_fwd(*args, h0=st["h0"], lengths=st["lengths"])
    y, _, states = ssm.gdr_fwd(*args, lengths=st["lengths"], return_h_last=False, return_states=True)
    return (y,) + tuple(ssm.gdr_bwd(*args, states, st["dy"], lengths=st["lengths"], return_dh0=False)[:5])


def _own_qkn(st):
    import state_space_model_ssm_amd as ssm
    kw = dict(inv_freq=st["inv_freq"], pos=st["pos"], eps=EPS, neighbours=st["pairs"] == "neighbours")
    out = ssm.qk_norm_fwd(st["q"], st["k"], st["wq"], st["wk"], **kw)
    if st["dir"] == "fwd":
        return out
    dq, dk, dwq, dwk = ssm.qk_norm_bwd(st["q"], st["k"], st["wq"], st["wk"], st["dq"], st["dk"], **kw)
    return (*out, dq, dwq, dk, dwk)


def _own_swa8(st):
    import state_space_model_ssm_amd as ssm
    cache = ssm.SwaQ8Cache(*st["cache"])
    if st["dir"] == "fill":
        ssm.swa_q8_fill(st["k"], st["v"], cache, sinks=st["sinks"], lengths=st["lengths"])
        return tuple(st["cache"])
    y = ssm.swa_q8_step(st["q"], st["k"], st["v"], cache, st["pos"], sinks=st["sinks"])
    return (y, *st["cache"])


def run(st):
    plain, kernels = {"gdr": (_plain_gdr, _own_gdr), "qkn": (_plain_qkn, _own_qkn),
                      "swa8": (_plain_swa8, _own_swa8)}[st["op"]]
    return kernels(st) if own else plain(st)


# ---------------------------------------------------------------------------
# Bytes and operations
# ---------------------------------------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    train = case["dir"] == "train"
    if case["op"] == "gdr":
        kd, vd, h = case["kdim"], case["vdim"], case["heads"]
        # Rows of unequal length have 5/8 of the longest's tokens on average.
        tokens = case["batch"] * case["seqlen"] * (0.625 if case["ragged"] else 1.0)
        states = 4 * case["batch"] * h * kd * vd * (2 if case["state"] else 0 if train else 1)
        each = e * (2 * case["qk_heads"] * kd + h * vd) + 2 * h * (2 if case["gates"] == "bf16" else 4)
        return {"bytes": tokens * (each * (2 if train else 1) + e * h * vd * (2 if train else 1)) + states,
                "flops": tokens * h * kd * vd * (20 if train else 6)}
    h, kv, d = case["heads"], case["kv_heads"], case["headdim"]
    if case["op"] == "qkn":
        n = case["batch"] * case["seqlen"] * (h + kv) * d
        return {"bytes": n * e * (4 if train else 2), "flops": n * (24 if train else 8)}
    window, part = case["window"], 0.75 if case["ragged"] else 1.0
    if case["dir"] == "step":
        keys = case["batch"] * (window * part + case["sinks"])
        return {"bytes": 2 * d * kv * keys * (1 + 4 / (BLOCK * d)) + 2 * d * case["batch"] * (2 * h + 2 * kv),
                "flops": 4 * d * h * keys}
    tokens = case["batch"] * min(window + case["sinks"], case["seqlen"] * (0.625 if case["ragged"] else 1.0))
    return {"bytes": 2 * tokens * kv * d * 3, "flops": 2 * tokens * kv * d * 4}


# ---------------------------------------------------------------------------
# The definitions in float64
# ---------------------------------------------------------------------------

def _exact_gdr(st):
    step, train = st["dir"] == "step", st["dir"] == "train"
    q, k, v, g, beta = (st[t].double().unsqueeze(1) if step else st[t].double() for t in ("q", "k", "v", "g", "beta"))
    b, n, h, vd = v.shape
    qk, kd = q.shape[2:]
    share, scale = h // qk, kd ** -0.5
    q, k = (t.unsqueeze(3).expand(b, n, qk, share, kd).reshape(b, n, h, kd) for t in (q, k))
    if st["lengths"] is not None:
        for row, m in enumerate(st["lengths"].tolist()):
            g[row, m:], beta[row, m:], q[row, m:] = 0, 0, 0
    a = torch.exp(g)
    s = torch.zeros(b, h, vd, kd, dtype=torch.float64, device=v.device) if st["h0"] is None else st["h0"].double()
    y = torch.empty_like(v)
    past = [s] if train else None
    for t in range(n):
        kt, at = k[:, t, :, :, None], a[:, t, :, None]
        u = beta[:, t, :, None] * (v[:, t] - at * (s @ kt)[..., 0])
        s = torch.baddbmm((at[..., None] * s).view(b * h, vd, kd), u.reshape(b * h, vd, 1),
                          k[:, t].reshape(b * h, 1, kd)).view(b, h, vd, kd)
        y[:, t] = (s @ q[:, t, :, :, None])[..., 0] * scale
        if train:
            past.append(s)
    if not train:
        return (y[:, 0], s) if step else (y, s)
    dq, dk, dv, dg, db = (torch.zeros_like(t) for t in (q, k, v, g, beta))
    dy = st["dy"].double()
    if st["lengths"] is not None:
        for row, m in enumerate(st["lengths"].tolist()):
            dy[row, m:] = 0
    ds = torch.zeros_like(s)
    for t in range(n - 1, -1, -1):
        s, at, bt, kt, before = past.pop(), a[:, t], beta[:, t], k[:, t], past[-1]
        ds = ds + scale * dy[:, t, :, :, None] * q[:, t, :, None, :]
        dq[:, t] = scale * (dy[:, t, :, None, :] @ s)[:, :, 0]
        seen = (before @ kt[..., None])[..., 0]
        rest = v[:, t] - at[..., None] * seen
        du = (ds @ kt[..., None])[..., 0]
        db[:, t] = (du * rest).sum(-1)
        dv[:, t] = bt[..., None] * du
        dk[:, t] = ((bt[..., None] * rest)[:, :, None] @ ds)[:, :, 0] - at[..., None] * (dv[:, t, :, None] @ before)[:, :, 0]
        dg[:, t] = at * ((ds * before).sum((-1, -2)) - (dv[:, t] * seen).sum(-1))
        ds = at[..., None, None] * (ds - dv[:, t, :, :, None] * kt[:, :, None])
    if st["lengths"] is not None:
        for row, m in enumerate(st["lengths"].tolist()):
            dk[row, m:], dg[row, m:], db[row, m:] = 0, 0, 0
    dq, dk = (t.unflatten(2, (qk, share)).sum(3) for t in (dq, dk))
    return y, dq, dk, dv, dg, db


def _exact_qkn(st):
    half = st["inv_freq"].shape[0]
    angle = st["pos"].double().unsqueeze(-1) * st["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(2)
    outs, grads = [], []
    for name in ("q", "k"):
        x = st[name].double().requires_grad_(True)
        w = st["w" + name].double().requires_grad_(True)
        n = w * x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
        head, rest = n[..., :2 * half], n[..., 2 * half:]
        halves = st["pairs"] == "halves"
        z = torch.complex(head[..., :half], head[..., half:]) if halves else torch.complex(head[..., ::2], head[..., 1::2])
        z = z * turn
        z = torch.cat([z.real, z.imag], -1) if halves else torch.view_as_real(z).flatten(-2)
        out = torch.cat([z, rest], -1)
        outs.append(out.detach())
        if st["dir"] == "train":
            grads += list(torch.autograd.grad(out, (x, w), st["d" + name].double()))
    return tuple(outs + grads)


def _exact_blocks(x):
    """x / scale and the scale, of (kv, block, d)."""
    top = x.double().abs().flatten(1).max(1).values / 448
    return x.double() / torch.where(top > 0, top, 1.0)[:, None, None], top


def _exact_swa8(st):
    window, sinks = st["window"], st["sinks"]
    near, ring, scale = ([t.double() for t in st["cache"][i:i + 2]] for i in (0, 2, 4))
    b, kv = near[0].shape[:2]
    d = near[0].shape[-1]
    new = (st["k"], st["v"])
    if st["dir"] == "fill":
        for row in range(b):
            m = st["k"].shape[1] if st["lengths"] is None else int(st["lengths"][row])
            for x, nr, rg, sc in zip(new, near, ring, scale):
                nr[row, :, :min(m, sinks)] = x[row, :min(m, sinks)].transpose(0, 1).double()
                whole = max(0, m - sinks) // BLOCK
                left = max(0, m - sinks) - whole * BLOCK
                nr[row, :, sinks:sinks + left] = x[row, m - left:m].transpose(0, 1).double()
                for blk in range(max(0, whole - window // BLOCK), whole):
                    at, spot = sinks + blk * BLOCK, blk % (window // BLOCK)
                    q, s = _exact_blocks(x[row, at:at + BLOCK].transpose(0, 1))
                    rg[row, :, spot * BLOCK:(spot + 1) * BLOCK], sc[row, :, spot] = q, s
        return (*near, *ring, *scale)
    y = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    group = y.shape[1] // kv
    for row, p in enumerate(st["pos"].tolist()):
        off = (p - sinks) % BLOCK
        for x, nr in zip(new, near):
            nr[row, :, p if p < sinks else sinks + off] = x[row].double()
        # The position that every place of the cache holds now, or -1.
        where = [j if j <= p else -1 for j in range(sinks)]
        first = p - off
        where += [first + j if p >= sinks and j <= off else -1 for j in range(BLOCK)]
        for s in range(window):
            j = sinks + s
            if p >= j:
                j += (p - j) // window * window
            where.append(j if j <= p and j < first else -1)
        sel = torch.tensor([j >= 0 for j in where], device="cuda")
        keys, values = (torch.cat([nr[row], rg[row] * sc[row].repeat_interleave(BLOCK, 1)[..., None]], 1)[:, sel]
                        for nr, rg, sc in zip(near, ring, scale))
        for c in range(kv):
            s = st["q"][row, c * group:(c + 1) * group].double() @ keys[c].T / math.sqrt(d)
            y[row, c * group:(c + 1) * group] = torch.softmax(s, 1) @ values[c]
        if p >= sinks and off == BLOCK - 1:
            spot = (p - sinks) % window // BLOCK
            for nr, rg, sc in zip(near, ring, scale):
                q, s = _exact_blocks(nr[row, :, sinks:])
                rg[row, :, spot * BLOCK:(spot + 1) * BLOCK], sc[row, :, spot] = q, s
    return (y, *near, *ring, *scale)


def exact(case, seed):
    return {"gdr": _exact_gdr, "qkn": _exact_qkn, "swa8": _exact_swa8}[case["op"]](prepare(case, seed))
