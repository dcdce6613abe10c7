"""libssm_delta on the host: the library loads, exports exactly what
include/ssm_delta.h declares, and rejects every bad request before any HIP
call (the fake device addresses below are never dereferenced); the binding
rejects mis-shaped arguments before any call into the library."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import delta_reference as ref
import state_space_model_ssm_amd as ssm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssm_delta.h")
FAKE = 0x7F0000000000
needs_no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="fake device pointers must never reach a GPU")

OK, NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3, -4, -5, -6


def at(k):
    """Fake addresses 1 TiB apart: no two tensors meet."""
    return FAKE + (k << 40)


def gdr(**kw):
    d = dict(batch=8, seqlen=200, nqk=2, nheads=4, kdim=64, vdim=128, q_batch=200 * 128, q_token=128, k_batch=200 * 128,
             k_token=128, v_batch=200 * 512, v_token=512, scale=0.125, gate_dtype=1, workspace=at(50),
             workspace_bytes=1 << 40)
    return ssm.GdrDims(**{**d, **kw})


def qkn(**kw):
    d = dict(batch=2, seqlen=20, nheads=4, nkv=2, headdim=64, rot=64, q_batch=20 * 256, q_token=256, k_batch=20 * 128,
             k_token=128, oq_batch=20 * 256, oq_token=256, ok_batch=20 * 128, ok_token=128, dtype=1, neighbours=0, eps=1e-6,
             workspace=at(50), workspace_bytes=1 << 40)
    return ssm.QkNormDims(**{**d, **kw})


def swa(**kw):
    d = dict(batch=8, seqlen=40, nheads=4, nkv=2, headdim=64, window=128, sinks=2, q_batch=40 * 256, q_token=256,
             k_batch=40 * 128, k_token=128, v_batch=40 * 128, v_token=128, scale=0.125, workspace=at(50),
             workspace_bytes=1 << 40)
    return ssm.SwaDims(**{**d, **kw})


def one(make):
    return lambda **kw: make(**{**dict(seqlen=1), **kw})


CALLS = {  # entry point: (dims, pointers, required ones, outputs)
    "ssm_gdr_fwd": (gdr, 10, (0, 1, 2, 3, 4, 7), (7, 8, 9)),
    "ssm_gdr_bwd": (gdr, 12, (0, 1, 3, 4, 6, 7, 8, 9, 10), (6, 7, 8, 9, 10, 11)),
    "ssm_gdr_step": (one(gdr), 8, tuple(range(8)), (6, 7)),
    "ssm_qk_norm_fwd": (qkn, 8, (0, 1, 4, 6, 7), (6, 7)),
    "ssm_qk_norm_bwd": (qkn, 12, (0, 1, 4, 6, 7, 8, 9), (8, 9, 10, 11)),
    "ssm_swa_q8_step": (one(swa), 11, tuple(range(11)), (3, 4, 5, 6, 7, 8, 10)),
    "ssm_swa_q8_fill": (swa, 9, (0, 1, 3, 4, 5, 6, 7, 8), (3, 4, 5, 6, 7, 8)),
}
SIZES = {"ssm_gdr_workspace_size": gdr, "ssm_gdr_states_size": gdr, "ssm_gdr_bwd_workspace_size": gdr,
         "ssm_qk_norm_bwd_workspace_size": qkn, "ssm_swa_q8_step_workspace_size": one(swa)}


def call(name, pointers=None, **kw):
    args = [at(k) for k in range(CALLS[name][1])]
    for k, v in (pointers or {}).items():
        args[k] = v
    return getattr(ssm.delta_lib(), name)(*args, ctypes.byref(CALLS[name][0](**kw)), None)


def size(name, dims):
    n = ctypes.c_size_t(0)
    rc = getattr(ssm.delta_lib(), name)(ctypes.byref(dims), ctypes.byref(n))
    return rc if rc else n.value


def test_exports_exactly_the_header():
    text = open(HEADER).read()
    declared = sorted(set(re.findall(r"^SSM_API\s+[\w\s\*]*?\b(\w+)\s*\(", text, re.M)))
    out = os.popen(f"nm -D --defined-only {ssm.delta_library_path()}").read()
    assert sorted({l.split()[-1] for l in out.splitlines() if " T " in l}) == declared and len(declared) == 13
    assert set(CALLS) | set(SIZES) | {"ssm_delta_last_error"} == set(declared)


def test_struct_layouts_match_the_header(tmp_path):
    c = '#include <stdio.h>\n#include <stddef.h>\n#include "ssm_delta.h"\nint main(void) {\n'
    want = []
    for cname, t in (("ssm_gdr_dims_t", ssm.GdrDims), ("ssm_qk_norm_dims_t", ssm.QkNormDims)):
        c += f'printf("%zu\\n", sizeof({cname}));\n'
        want.append(ctypes.sizeof(t))
        for f in t._fields_:
            c += f'printf("%zu\\n", offsetof({cname}, {f[0]}));\n'
            want.append(getattr(t, f[0]).offset)
    src = tmp_path / "t.c"
    src.write_text(c + 'printf("%d\\n", SSM_GDR_STATE_STEP);\nreturn 0; }\n')
    exe = str(tmp_path / "t")
    subprocess.check_call(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe])
    assert [int(v) for v in subprocess.check_output([exe]).split()] == want + [ssm.GDR_STATE_STEP]


@needs_no_gpu
@pytest.mark.parametrize("name", CALLS)
def test_missing_and_misaligned_pointers(name):
    _, n, required, _ = CALLS[name]
    assert getattr(ssm.delta_lib(), name)(*[at(k) for k in range(n)], None, None) == NULL
    for k in required:
        assert call(name, pointers={k: None}) == NULL, k
        assert "required" in ssm.delta_last_error()
    for k in range(n):
        assert call(name, pointers={k: at(k) + 1}) == ALIGN, k
        assert "aligned" in ssm.delta_last_error()


@needs_no_gpu
@pytest.mark.parametrize("name", CALLS)
def test_overlaps(name):
    """Every output shifted by 16 bytes onto every other tensor of the call, which may be no output's exact place but the documented one."""
    exact = {("ssm_gdr_fwd", 8): 5, ("ssm_gdr_step", 7): 5, ("ssm_qk_norm_fwd", 6): 0, ("ssm_qk_norm_fwd", 7): 1,
             ("ssm_qk_norm_bwd", 8): 0, ("ssm_qk_norm_bwd", 9): 1}
    _, n, _, outs = CALLS[name]
    for o in outs:
        for k in range(n):
            if k != o:
                assert call(name, pointers={o: at(k) + 16}) == SHAPE, (o, k)
                assert "overlaps" in ssm.delta_last_error()
                if exact.get((name, o)) != k:
                    assert call(name, pointers={o: at(k)}) == SHAPE, (o, k)
    if name in ("ssm_gdr_fwd", "ssm_gdr_bwd", "ssm_qk_norm_bwd", "ssm_swa_q8_step"):
        assert call(name, pointers={outs[0]: at(50) + 16}) == SHAPE


@needs_no_gpu
@pytest.mark.parametrize("name,kw", [("ssm_gdr_fwd", {}), ("ssm_gdr_bwd", {}), ("ssm_qk_norm_bwd", {}),
                                     ("ssm_swa_q8_step", dict(window=8192))])
def test_workspaces(name, kw):
    """One that is missing, a byte short, misaligned, or over an input."""
    _, n, _, outs = CALLS[name]
    need = size(name.replace("_fwd", "") + "_workspace_size", CALLS[name][0](**kw))
    assert need > 0
    assert call(name, workspace_bytes=need - 1, **kw) == WORKSPACE and call(name, workspace=None, **kw) == WORKSPACE
    assert call(name, workspace=at(50) + 16, **kw) == ALIGN
    for k in range(n):
        if k not in outs:
            assert call(name, pointers={k: at(50) + 256}, workspace_bytes=need, **kw) == SHAPE, k
            assert "workspace overlaps" in ssm.delta_last_error()


@needs_no_gpu
@pytest.mark.parametrize("name", SIZES)
def test_sizes_of_nothing(name):
    f, n = getattr(ssm.delta_lib(), name), ctypes.c_size_t()
    assert f(ctypes.byref(SIZES[name]()), None) == NULL and f(None, ctypes.byref(n)) == NULL
    assert size(name, SIZES[name](batch=-1)) == SHAPE


@needs_no_gpu
def test_gdr_sizes():
    for name in ("ssm_gdr_fwd", "ssm_gdr_bwd", "ssm_gdr_step"):
        assert call(name, batch=-1) == SHAPE and call(name, nqk=3) == SHAPE and call(name, nheads=0, nqk=0) == SHAPE
        assert call(name, kdim=32) == UNSUPPORTED and call(name, vdim=96) == UNSUPPORTED and call(name, vdim=256) == UNSUPPORTED
        assert call(name, gate_dtype=2) == DTYPE
        for scale in (math.nan, math.inf):
            assert call(name, scale=scale) == SHAPE
        for axis in ("q_batch", "k_batch", "v_batch", "q_token", "k_token", "v_token"):
            assert call(name, **{axis: 4}) == SHAPE and call(name, **{axis: -8}) == SHAPE
            assert call(name, **{axis: (1 << 40) + 8}) == SHAPE
        for axis in ("q_batch", "k_batch", "v_batch"):
            assert call(name, **{axis: 64}) == SHAPE and "smaller" in ssm.delta_last_error()
        assert call(name, batch=1 << 22) == UNSUPPORTED and call(name, batch=1 << 62) == UNSUPPORTED
        assert call(name, batch=0, nheads=1 << 62, nqk=1 << 62) == UNSUPPORTED
        wide = dict(batch=1, seqlen=1, nheads=1 << 18, nqk=1, v_batch=0, v_token=0)   # 2^25 elements a token
        assert call(name, **wide) == UNSUPPORTED and "2^24" in ssm.delta_last_error()
    for name in ("ssm_gdr_fwd", "ssm_gdr_bwd"):
        assert call(name, seqlen=-1) == SHAPE and call(name, seqlen=(1 << 30) + 1) == UNSUPPORTED
        assert call(name, batch=1, nheads=1, nqk=1, seqlen=1 << 30) == UNSUPPORTED   # 2^24 blocks of 64 tokens
        for axis in ("q_token", "k_token", "v_token"):
            assert call(name, **{axis: 56}) == SHAPE
            far = (1 << 24) + 8
            assert call(name, batch=1, **{axis: far}) == UNSUPPORTED
    assert call("ssm_gdr_step", seqlen=2) == SHAPE and call("ssm_gdr_step", seqlen=0) == SHAPE
    # Per value head and 64 tokens: the state, the u_t, and what of v and the gates the backward needs.
    assert size("ssm_gdr_states_size", gdr(seqlen=129)) == 8 * 4 * 3 * (4 * 128 * (64 + 64) + 26624)
    assert size("ssm_gdr_states_size", gdr(seqlen=0)) == 0 == size("ssm_gdr_states_size", gdr(batch=0))


@needs_no_gpu
def test_segments_stay_within_what_is_launched():
    """A long sequence of few heads is cut into segments, each with a state of its own: at most 64 of them and 512
    workgroups' worth, and the workspace grows by that and no more."""
    for batch in (1, 2, 5, 33, 64, 300):
        for nheads, nqk in ((1, 1), (3, 1), (16, 4), (64, 64)):
            for seqlen in (0, 1, 63, 64, 65, 640, 4096, 4097, 65536, 1 << 20):
                for kdim, vdim in ((64, 64), (128, 128)):
                    d = gdr(batch=batch, nheads=nheads, nqk=nqk, seqlen=seqlen, kdim=kdim, vdim=vdim, q_token=nqk * kdim,
                            k_token=nqk * kdim, v_token=nheads * vdim, q_batch=1 << 40, k_batch=1 << 40, v_batch=1 << 40)
                    heads, chunks = batch * nheads, -(-seqlen // 64)
                    if heads * max(4, chunks) >= 1 << 24:
                        assert size("ssm_gdr_workspace_size", d) == UNSUPPORTED
                        continue
                    segments = max(1, min(64, chunks, 512 // (heads * vdim // 32)))
                    each = 4 * vdim * kdim + 4 * kdim * kdim
                    need = size("ssm_gdr_workspace_size", d)
                    if segments == 1:   # the blocks' parts alone
                        assert need % max(1, heads * chunks) == 0
                    assert 0 <= need <= heads * chunks * (1 << 17) + heads * segments * each
                    assert size("ssm_gdr_bwd_workspace_size", d) <= heads * chunks * (1 << 18) + heads * segments * each


@needs_no_gpu
def test_qk_norm_sizes():
    for name in ("ssm_qk_norm_fwd", "ssm_qk_norm_bwd"):
        assert call(name, batch=-1) == SHAPE and call(name, seqlen=-1) == SHAPE and call(name, nheads=0) == SHAPE
        assert call(name, nkv=0) == SHAPE and call(name, headdim=24, rot=0) == UNSUPPORTED and call(name, headdim=272) == UNSUPPORTED
        assert call(name, rot=8) == SHAPE and call(name, rot=80) == SHAPE and call(name, rot=-16) == SHAPE
        assert call(name, dtype=2) == DTYPE and call(name, neighbours=2) == SHAPE and call(name, reserved=1) == SHAPE
        for eps in (-1e-6, math.nan, math.inf):
            assert call(name, eps=eps) == SHAPE
        assert call(name, nheads=(1 << 20) + 1) == UNSUPPORTED and call(name, seqlen=1 << 31) == UNSUPPORTED
        assert call(name, batch=1 << 60) == UNSUPPORTED
        for axis in ("q_batch", "q_token", "k_batch", "k_token", "oq_batch", "oq_token", "ok_batch", "ok_token"):
            assert call(name, **{axis: 4}) == SHAPE and call(name, **{axis: -8}) == SHAPE and call(name, **{axis: 64}) == SHAPE
        # Rows far apart: refused before a product of sizes overflows.
        far = 1 << 40
        assert call(name, batch=1 << 30, q_batch=far) == UNSUPPORTED
        assert call(name, batch=1, seqlen=1 << 30, oq_token=far, ok_token=far) == UNSUPPORTED
        # Rows of an output that meet; batch and token strides may change places.
        assert call(name, oq_batch=512) == SHAPE and "overlap" in ssm.delta_last_error()
        assert call(name, batch=0, oq_batch=256, oq_token=512, pointers={10: None, 11: None} if name.endswith("bwd") else {}) == OK
    assert call("ssm_qk_norm_fwd", pointers={4: None}, rot=0, batch=0) == OK
    # q and k as parts of one projection, in place: side by side, and one element into each other.
    side = dict(q_batch=20 * 384, q_token=384, k_batch=20 * 384, k_token=384, oq_batch=20 * 384, oq_token=384,
                ok_batch=20 * 384, ok_token=384)
    for k in (at(0) + 2 * 248, at(0) + 2 * 264):
        assert call("ssm_qk_norm_fwd", pointers={1: k, 6: at(0), 7: k}, **side) == SHAPE
        assert "overlaps" in ssm.delta_last_error()


@needs_no_gpu
def test_swa_q8_sizes():
    for name in ("ssm_swa_q8_step", "ssm_swa_q8_fill"):
        assert call(name, batch=-1) == SHAPE and call(name, nkv=3) == SHAPE and call(name, nheads=0, nkv=0) == SHAPE
        for window in (0, 32, 65, 100):
            assert call(name, window=window) == SHAPE
        assert call(name, sinks=-1) == SHAPE and call(name, headdim=96) == UNSUPPORTED
        assert call(name, window=1 << 30, sinks=64) == UNSUPPORTED and call(name, window=1 << 31) == UNSUPPORTED
        assert call(name, batch=1 << 20) == UNSUPPORTED and call(name, scale=math.nan) == SHAPE
        assert call(name, k_batch=-8) == SHAPE and call(name, v_batch=8) == SHAPE and call(name, reserved=7) == SHAPE
    assert call("ssm_swa_q8_step", seqlen=2) == SHAPE
    assert call("ssm_swa_q8_fill", seqlen=1 << 31) == UNSUPPORTED and call("ssm_swa_q8_fill", k_token=64) == SHAPE
    for batch, nheads, nkv in ((1, 1, 1), (1, 128, 1), (64, 32, 8), (1000, 40, 5), (65535, 1, 1)):
        for window in (64, 4096, 1 << 20, 1 << 29):
            d = swa(seqlen=1, batch=batch, nheads=nheads, nkv=nkv, window=window, headdim=128, q_batch=1 << 20, k_batch=1 << 20,
                    v_batch=1 << 20)
            # At most 1024 workgroups and one more per block of 16 heads, each with 16 heads' sums, a maximum and a sum.
            blocks = batch * nkv * -(-(nheads // nkv) // 16)
            assert 0 <= size("ssm_swa_q8_step_workspace_size", d) <= (1024 + blocks) * 16 * (128 + 2) * 4 + 512


@needs_no_gpu
def test_empty_calls_launch_nothing():
    assert call("ssm_gdr_fwd", batch=0) == OK and ssm.delta_last_error() == ""
    assert call("ssm_gdr_fwd", seqlen=0, pointers={8: None}) == OK and call("ssm_gdr_bwd", seqlen=0, pointers={11: None}) == OK
    assert call("ssm_gdr_bwd", batch=0) == OK and call("ssm_gdr_step", batch=0) == OK
    assert call("ssm_qk_norm_fwd", batch=0) == OK and call("ssm_qk_norm_fwd", seqlen=0) == OK
    assert call("ssm_qk_norm_bwd", seqlen=0, pointers={10: None, 11: None}) == OK
    assert call("ssm_swa_q8_step", batch=0) == OK and call("ssm_swa_q8_fill", seqlen=0) == OK
    assert call("ssm_swa_q8_fill", batch=0) == OK


def test_binding_refuses_before_the_library():
    z = torch.zeros
    b = lambda *s: z(*s, dtype=torch.bfloat16)
    q, v, g = b(2, 5, 2, 64), b(2, 5, 4, 64), z(2, 5, 4)
    with pytest.raises(ValueError, match="on the GPU"):
        ssm.gdr_fwd(q, q, v, g, g)
    with pytest.raises(ValueError, match="on the GPU"):
        ssm.gdr_step(q[:, 0], q[:, 0], v[:, 0], g[:, 0], g[:, 0], z(2, 4, 64, 64))
    with pytest.raises(ValueError, match="on the GPU"):
        ssm.gdr_bwd(q, q, v, g, g, z(8, dtype=torch.uint8), v)
    with pytest.raises(ValueError, match="on the GPU"):
        ssm.qk_norm_fwd(q, q)
    with pytest.raises(ValueError, match="on the GPU"):
        ssm.qk_norm_bwd(q, q, None, None, q, q)
    cache = ssm.swa_q8_cache(2, 2, 64, 64, sinks=1, device="cpu")
    assert [tuple(t.shape) for t in cache] == [(2, 2, 65, 64)] * 2 + [(2, 2, 64, 64)] * 2 + [(2, 2, 1)] * 2
    with pytest.raises(ValueError, match="on the GPU"):
        ssm.swa_q8_step(q[:, 0], q[:, 0], q[:, 0], cache, z(2), sinks=1)
    with pytest.raises(ValueError, match="on the GPU"):
        ssm.swa_q8_fill(q, q, cache, sinks=1)
    for window in (0, 63, 100):
        with pytest.raises(ValueError, match="multiple of 64"):
            ssm.swa_q8_cache(1, 1, window, 64, device="cpu")


def test_the_float64_forms_catch_planted_mistakes():
    """The plain forms agree with others written another way, and a mistake in either shows."""
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    q, k, v = r(1, 9, 1, 6), r(1, 9, 1, 6), r(1, 9, 2, 5)
    k = k / k.norm(dim=-1, keepdim=True)
    g, beta, h0 = -torch.rand(1, 9, 2, generator=gen).double(), torch.rand(1, 9, 2, generator=gen).double(), r(1, 2, 5, 6)
    leaves = [t.requires_grad_() for t in (q, k, v, g, beta, h0)]
    y, last, _, _ = ref.gdr(*leaves)
    for h in range(2):   # S_t = S_{t-1} a (I - beta k k^T) + beta v k^T, as products of matrices
        S = h0[0, h]
        for t in range(9):
            kt, b = k[0, t, 0], beta[0, t, h]
            S = torch.exp(g[0, t, h]) * S @ (torch.eye(6, dtype=torch.float64) - b * torch.outer(kt, kt)) + b * torch.outer(v[0, t, h], kt)
            assert torch.allclose(y[0, t, h], S @ q[0, t, 0] * 6 ** -0.5, rtol=1e-10)
        assert torch.allclose(last[0, h], S, rtol=1e-10)
    dy, dl = r(1, 9, 2, 5), r(1, 2, 5, 6)
    want = torch.autograd.grad((y * dy).sum() + (last * dl).sum(), leaves)
    plain = [t.detach() for t in leaves]
    got = ref.gdr_bwd(*plain[:5], dy, plain[5], dh_last=dl)[0]
    for name, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), want):
        assert torch.allclose(got[name], w, rtol=1e-9, atol=1e-12), name
    wrong = ref.gdr_bwd(*plain[:5], dy, plain[5])[0]   # without the state's own gradient
    assert not any(torch.allclose(wrong[n], got[n], rtol=1e-3) for n in ("dk", "dv", "dg", "dbeta", "dh0"))
    assert not torch.allclose(ref.gdr(*plain[:4], plain[4] * 1.01, plain[5])[0], y.detach(), rtol=1e-4)

    x, w, f = r(1, 3, 2, 16), r(16), torch.tensor([0.5, 0.25, 0.125, 0.0625], dtype=torch.float32)
    pos = torch.tensor([[0, 1, 7]], dtype=torch.int32)
    for nb in (False, True):
        out = ref.qk_norm(x, w, f, pos, 1e-6, nb)
        n = x / torch.sqrt((x * x).sum(-1, keepdim=True) / 16 + 1e-6) * w
        for t in range(3):
            for i in range(4):
                a, c = (2 * i, 2 * i + 1) if nb else (i, i + 4)
                z = torch.complex(n[0, t, :, a], n[0, t, :, c]) * torch.polar(torch.tensor(1.0).double(), pos[0, t].double() * f[i].double())
                assert torch.allclose(out[0, t, :, a], z.real) and torch.allclose(out[0, t, :, c], z.imag)
        assert torch.equal(out[..., 8:], n[..., 8:])
        assert not torch.allclose(out, ref.qk_norm(x, w, f, pos, 1e-6, not nb))

    values = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    own = torch.unique(values.float()[~values.float().isnan()].abs().double())
    assert torch.equal(own, ref.E4M3) and len(own) == 127
    some = torch.cat([r(4096) * 100, ref.E4M3, (ref.E4M3[1:] + ref.E4M3[:-1]) / 2]).clamp(-448, 448)
    assert torch.equal(ref.to_e4m3(some), some.float().to(torch.float8_e4m3fn).double())
    model = ref.Q8Cache(1, 1, 64, 2, 1)
    for t in range(2):
        model.rows[0][t].extend(r(1, 2) for _ in range(200))
    pos = 150   # blocks 1 .. 64 and 65 .. 128 are whole; seen: the sink and the last 64
    held = model.held(0, 0, pos)
    raw = torch.stack(model.rows[0][0])
    assert held.shape == (65, 1, 2) and torch.equal(held[0], raw[0]) and torch.equal(held[-22:], raw[129:151])
    off = (held[1:-22] - raw[87:129]).abs()
    assert 0 < off.max() <= raw[65:129].abs().max() / 448 * 16   # half a step of the largest numbers
