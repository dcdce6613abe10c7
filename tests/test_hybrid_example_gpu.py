"""The hybrid block example: its gradients against a plain float64 model, its
decoding against the whole sequence, and its training."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_block.py")
    spec = importlib.util.spec_from_file_location("hybrid_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain(model, p, tokens, lengths, reset):
    """The example's logits in float64 from parameters p, with torch's own operators."""
    L = tokens.shape[1]
    x, s = p["embed.weight"][tokens], 0.0

    def norm(x, s, w):
        s = x + s
        return s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-5) * w, s

    t = torch.arange(L)
    for n, mixer in enumerate(model.mixers):
        y, s = norm(x, s, p[f"norms.{n}"])
        w = {k.split(".", 2)[2]: v for k, v in p.items() if k.startswith(f"mixers.{n}.")}
        if "log_a" in w:
            u, rec, inp = (y @ w[f"{k}.weight"].T for k in ("x", "rec", "inp"))
            a = torch.exp(-torch.exp(w["log_a"]) * torch.sigmoid(rec))
            u = torch.sqrt(1 - a * a) * torch.sigmoid(inp) * u
            h, out = torch.zeros_like(u[:, 0]), []
            for i in range(L):
                h = a[:, i] * torch.where(reset[:, i, None], 0.0, h) + u[:, i]
                out.append(h)
            x = torch.stack(out, 1) @ w["out.weight"].T
        else:
            H, KV, _ = mixer.split
            q, k, v = (y @ w["qkv.weight"].T).unflatten(-1, (-1, mixer.headdim)).split(mixer.split, -2)
            k, v = (z.repeat_interleave(H // KV, 2) for z in (k, v))
            gap = t[:, None] - t[None]
            see = (gap >= 0) & ((gap < mixer.window) | (t[None] < mixer.sinks))
            see = see[None] & (t[None, None] < lengths[:, None, None])
            sc = torch.einsum("bthd,bjhd->bhtj", q, k) * mixer.headdim ** -0.5
            pr = torch.softmax(sc.masked_fill(~see[:, None], float("-inf")), -1)
            o = torch.einsum("bhtj,bjhd->bthd", pr, v) * (t[None] < lengths[:, None])[..., None, None]
            x = o.flatten(-2) @ w["out.weight"].T
    return norm(x, s, p["norms.%d" % len(model.mixers)])[0] @ p["head.weight"].T


def test_gradients_against_a_plain_model(example):
    torch.manual_seed(0)
    model = example.HybridModel(vocab=40, dim=128, layers=1, heads=4, kv_heads=2, window=20, sinks=3).cuda()
    tokens = torch.randint(40, (3, 77))
    lengths = torch.tensor([77, 50, 1], dtype=torch.int32)
    reset = torch.rand(3, 77) < 0.05
    weight = torch.randn(3, 77, 40).double() * (torch.arange(77)[None] < lengths[:, None])[..., None]
    logits = model(tokens.cuda(), lengths.cuda(), reset.cuda())
    (logits.double() * weight.cuda()).sum().backward()
    p = {k: v.detach().cpu().double().requires_grad_() for k, v in model.named_parameters()}
    want = plain(model, p, tokens, lengths, reset)
    (want * weight).sum().backward()
    # Some 12 tensors on the way are rounded to bfloat16 (2^-9 each, of their own size), forward and back.
    bound = 24 * 2.0 ** -9
    seen = (torch.arange(77)[None] < lengths[:, None])
    assert float((logits.cpu().double() - want).detach()[seen].norm()) <= bound * float(want.detach()[seen].norm())
    for k, v in model.named_parameters():
        err = float((v.grad.cpu().double() - p[k].grad).norm() / p[k].grad.norm())
        assert err <= bound, (k, err)


@pytest.mark.parametrize("prompt", [1, 5, 63, 300])
def test_decoding_goes_on_where_the_prompt_ends(example, prompt):
    torch.manual_seed(1)
    model = example.HybridModel(layers=1, window=128).cuda()
    tokens = torch.randint(256, (3, prompt + 70), device="cuda")
    got = example.decode(model, tokens, prompt).float()
    with torch.no_grad():
        want = model(tokens)[:, prompt - 1:].float()
    # Two paths of some 12 roundings to 2^-9, and one to e4m3 (2^-4 of a value at most, half of it the
    # last place): the norm of their difference.
    assert float((got - want).norm()) <= (24 * 2.0 ** -9 + 2.0 ** -4) * float(want.norm())


def test_training_lowers_the_loss(example):
    torch.manual_seed(2)
    model = example.HybridModel(dim=256, layers=1, heads=4, window=64).cuda()
    losses = example.train(model, example.sequence(4, 200, 256, "cuda"), 20)
    assert all(l == l for l in losses) and losses[-1] < 0.8 * losses[0], losses
