"""The delta block example: its gradients against a plain float64 model, its
decoding against the whole sequence, alone and as a captured graph, and its
training's run."""
import importlib.util
import os

import pytest
import torch

import delta_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "delta_block.py")
    spec = importlib.util.spec_from_file_location("delta_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain(model, p, tokens, lengths):
    """The example's logits in float64 from parameters p."""
    L = tokens.shape[1]
    x, s = p["embed.weight"][tokens], 0.0

    def norm(x, s, w):
        s = x + s
        return s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-5) * w, s

    t = torch.arange(L)
    for n, mixer in enumerate(model.mixers):
        y, s = norm(x, s, p[f"norms.{n}"])
        w = {k.split(".", 2)[2]: v for k, v in p.items() if k.startswith(f"mixers.{n}.")}
        if "log_rate" in w:
            qk, v = (y @ w["proj.weight"].T).split(mixer.split, -1)
            q, k = qk.unflatten(-1, (-1, mixer.dims[0])).chunk(2, -2)
            q, k = (ref.qk_norm(z, mixer.dims[0] ** -0.5, None, None, 1e-6, False) for z in (q, k))
            decay, beta = (y @ w["gates.weight"].T).chunk(2, -1)
            g = -torch.exp(w["log_rate"]) * torch.nn.functional.softplus(decay)
            o = ref.gdr(q, k, v.unflatten(-1, (-1, mixer.dims[1])), g, torch.sigmoid(beta), lengths=lengths)[0]
        else:
            H, KV, _ = mixer.split
            q, k, v = (y @ w["qkv.weight"].T).unflatten(-1, (-1, mixer.headdim)).split(mixer.split, -2)
            pos, f = t[None].expand(len(tokens), -1), mixer.inv_freq.cpu()
            q, k = (ref.qk_norm(z, w[name], f, pos, 1e-6, False) for z, name in ((q, "wq"), (k, "wk")))
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
    model = example.DeltaModel(vocab=40, dim=128, layers=1, qk_heads=1, heads=2, kv_heads=1, window=20, sinks=3).cuda()
    tokens = torch.randint(40, (3, 77))
    lengths = torch.tensor([77, 50, 1], dtype=torch.int32)
    seen = torch.arange(77)[None] < lengths[:, None]
    weight = torch.randn(3, 77, 40).double() * seen[..., None]
    logits = model(tokens.cuda(), lengths.cuda())
    (logits.double() * weight.cuda()).sum().backward()
    p = {k: v.detach().cpu().double().requires_grad_() for k, v in model.named_parameters()}
    want = plain(model, p, tokens, lengths)
    (want * weight).sum().backward()
    # Some 14 tensors on the way are rounded to bfloat16 (2^-9 each, of their own size), forward and back.
    bound = 28 * 2.0 ** -9
    assert float((logits.cpu().double() - want).detach()[seen].norm()) <= bound * float(want.detach()[seen].norm())
    for k, v in model.named_parameters():
        err = float((v.grad.cpu().double() - p[k].grad).norm() / p[k].grad.norm())
        assert err <= bound, (k, err)


@pytest.mark.parametrize("prompt", [1, 5, 64, 300])
def test_decoding_goes_on_where_the_prompt_ends(example, prompt):
    torch.manual_seed(1)
    model = example.DeltaModel(layers=1, window=128).cuda()
    tokens = torch.randint(256, (3, prompt + 140), device="cuda")
    got = example.decode(model, tokens, prompt).float()
    with torch.no_grad():
        want = model(tokens)[:, prompt - 1:].float()
    # Two paths of some 14 roundings to 2^-9, and keys and values in e4m3 (2^-4 of a value at most, by
    # norms less): scores of normalised heads within 8 of each other move by 2^-4 / sqrt(3) of their spread.
    assert float((got - want).norm()) <= (28 * 2.0 ** -9 + 2.0 ** -4) * float(want.norm())


def test_decoding_as_a_captured_graph(example):
    """A step with its state, 8-bit cache and position in a graph, replayed token by token, gives what eager steps give."""
    torch.manual_seed(2)
    model = example.DeltaModel(layers=1, window=64).cuda()
    tokens = torch.randint(256, (2, 200), device="cuda")
    with torch.no_grad():
        _, eager = model.prefill(tokens[:, :50].contiguous())
        _, kept = model.prefill(tokens[:, :50].contiguous())
        token, pos = tokens[:, 50].contiguous(), torch.full((2,), 50, dtype=torch.int32, device="cuda")
        _, spare = model.prefill(tokens[:, :50].contiguous())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):   # the libraries' first calls, on states of no further use
            model.step(token, spare, pos)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            logits = model.step(token, kept, pos)
        at = torch.full_like(pos, 50)
        for i in range(50, 200):
            want = model.step(tokens[:, i].contiguous(), eager, at)
            token.copy_(tokens[:, i])
            pos.fill_(i)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(logits, want), i
            at += 1


def test_training_runs(example):
    torch.manual_seed(3)
    model = example.DeltaModel(dim=256, layers=1, heads=4, window=64).cuda()
    losses = example.train(model, example.sequence(2, 150, 256, "cuda"), 3)
    assert len(losses) == 3 and all(l == l and l < float("inf") for l in losses)
