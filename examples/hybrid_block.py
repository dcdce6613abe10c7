"""A hybrid language model's blocks on the operators of libssm_block: a gated
linear recurrence and sliding-window attention with sinks in turn, each after
a residual addition with RMS norm.

    python examples/hybrid_block.py [--steps 30] [--prompt 1000] [--tokens 64]

trains a small model on a synthetic sequence (forward and backward of all
three operators), reads a prompt in one pass, and goes on token by token from
the recurrence's states and the attention's ring caches, checking that the
tokens get the outputs the whole sequence would have given them.
"""
import argparse
import os
import sys
import time

import torch
from torch import nn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import state_space_model_ssm_amd as ssm  # noqa: E402

BF16 = torch.bfloat16


class AddNorm(torch.autograd.Function):
    """(norm of x + residual, x + residual)."""

    @staticmethod
    def forward(ctx, x, residual, w):
        y, s = ssm.rms_add_fwd(x, w, residual)
        ctx.save_for_backward(s, w)
        return y, s

    @staticmethod
    def backward(ctx, dy, ds):
        s, w = ctx.saved_tensors
        dx, dw = ssm.rms_add_bwd(dy.contiguous(), s, w, dres=ds.contiguous())
        return dx, dx, dw


class Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, rec, inp, A, reset):
        y, _, states = ssm.glr_fwd(x, rec, inp, A, reset=reset, return_h_last=False, return_states=True)
        ctx.save_for_backward(x, rec, inp, A, states, reset)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, rec, inp, A, states, reset = ctx.saved_tensors
        dx, drec, dinp, dA, _ = ssm.glr_bwd(x, rec, inp, A, states, dy.contiguous(), reset=reset, return_dh0=False)
        return dx, drec, dinp, dA, None


class Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, window, sinks, lengths):
        y, lse = ssm.swa_fwd(q, k, v, window=window, sinks=sinks, lengths=lengths)
        ctx.save_for_backward(q, k, v, y, lse, lengths)
        ctx.sees = dict(window=window, sinks=sinks)
        return y

    @staticmethod
    def backward(ctx, dy):
        q, k, v, y, lse, lengths = ctx.saved_tensors
        return *ssm.swa_bwd(q, k, v, y, lse, dy.contiguous(), lengths=lengths, **ctx.sees), None, None, None


class RecurrentMixer(nn.Module):
    def __init__(self, dim):
        super().__init__()
        self.x, self.rec, self.inp, self.out = (nn.Linear(dim, dim, bias=False, dtype=BF16) for _ in range(4))
        self.log_a = nn.Parameter(torch.linspace(-4.0, 1.0, dim))   # A = -exp(log_a): slow and fast channels

    def gates(self, x):
        return self.x(x), self.rec(x), self.inp(x), -torch.exp(self.log_a)

    def forward(self, x, lengths, reset):
        return self.out(Recurrence.apply(*self.gates(x), reset))

    def prefill(self, x):
        y, h = ssm.glr_fwd(*self.gates(x))
        return self.out(y), h

    def step(self, x, h, pos):
        return self.out(ssm.glr_step(*self.gates(x), h)[0])         # h is updated in place


class WindowMixer(nn.Module):
    def __init__(self, dim, heads, kv_heads, headdim, window, sinks):
        super().__init__()
        self.split = (heads, kv_heads, kv_heads)
        self.headdim, self.window, self.sinks = headdim, window, sinks
        self.qkv = nn.Linear(dim, sum(self.split) * headdim, bias=False, dtype=BF16)
        self.out = nn.Linear(heads * headdim, dim, bias=False, dtype=BF16)

    def parts(self, x):
        """q, k and v as views of one product: the operators take them as they are."""
        return self.qkv(x).unflatten(-1, (-1, self.headdim)).split(self.split, -2)

    def forward(self, x, lengths, reset):
        return self.out(Attention.apply(*self.parts(x), self.window, self.sinks, lengths).flatten(-2))

    def prefill(self, x):
        q, k, v = self.parts(x)
        y, _ = ssm.swa_fwd(q, k, v, window=self.window, sinks=self.sinks, return_lse=False)
        caches = tuple(torch.empty(x.shape[0], self.split[1], self.sinks + self.window, self.headdim, dtype=BF16,
                                   device=x.device) for _ in range(2))
        ssm.swa_fill(k, v, *caches, sinks=self.sinks)
        return self.out(y.flatten(-2)), caches

    def step(self, x, caches, pos):
        return self.out(ssm.swa_step(*self.parts(x), *caches, pos, sinks=self.sinks).flatten(-2))


class HybridModel(nn.Module):
    """Tokens -> logits: `layers` pairs of a recurrent and a window mixer."""

    def __init__(self, vocab=256, dim=512, layers=2, heads=8, kv_heads=2, headdim=64, window=256, sinks=4):
        super().__init__()
        self.embed = nn.Embedding(vocab, dim, dtype=BF16)
        self.mixers = nn.ModuleList()
        for _ in range(layers):
            self.mixers += [RecurrentMixer(dim), WindowMixer(dim, heads, kv_heads, headdim, window, sinks)]
        self.norms = nn.ParameterList(nn.Parameter(torch.ones(dim)) for _ in range(2 * layers + 1))
        self.head = nn.Linear(dim, vocab, bias=False, dtype=BF16)

    def forward(self, tokens, lengths=None, reset=None):
        """Logits of (batch, L) tokens, for training.  lengths: tokens of each
        row; reset: where a new document starts and the recurrence forgets."""
        x, s = self.embed(tokens), torch.zeros_like(self.embed.weight[:1]).expand(*tokens.shape, -1).contiguous()
        for norm, mixer in zip(self.norms, self.mixers):
            y, s = AddNorm.apply(x, s, norm)
            x = mixer(y, lengths, reset)
        return self.head(AddNorm.apply(x, s, self.norms[-1])[0])

    def _logits8(self, x, s):
        # The last norm in 8 bits with a scale per 128 values, as an 8-bit product would take it; here it is
        # spread out again for the head's bfloat16 weights.
        q, scale, _ = ssm.rms_add_q8_fwd(x, self.norms[-1], s, group=128)
        return self.head((q.float().unflatten(-1, (-1, 128)) * scale[..., None]).flatten(-2).to(BF16))

    @torch.no_grad()
    def prefill(self, tokens):
        """Logits of the prompt's last token, and the caches to go on from."""
        x, s, caches = self.embed(tokens), None, []
        for norm, mixer in zip(self.norms, self.mixers):
            y, s = ssm.rms_add_fwd(x, norm, s)
            x, cache = mixer.prefill(y)
            caches.append(cache)
        return self._logits8(x[:, -1].contiguous(), s[:, -1].contiguous()), caches

    @torch.no_grad()
    def step(self, token, caches, pos):
        """Logits after one token per row, (batch,), at positions pos (int32)."""
        x, s = self.embed(token), None
        for norm, mixer, cache in zip(self.norms, self.mixers, caches):
            y, s = ssm.rms_add_fwd(x, norm, s)
            x = mixer.step(y, cache, pos)
        return self._logits8(x, s)


def sequence(batch, length, vocab, device, seed=0):
    """Tokens that follow from the two before them, but for some noise."""
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(vocab, (batch, length), generator=g)
    noise = torch.rand(batch, length, generator=g) < 0.1
    for i in range(2, length):
        t[:, i] = torch.where(noise[:, i], t[:, i], (3 * t[:, i - 1] + t[:, i - 2] + 1) % vocab)
    return t.to(device)


def train(model, tokens, steps, lr=2e-3):
    opt = torch.optim.AdamW(model.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        logits = model(tokens[:, :-1].contiguous())
        loss = nn.functional.cross_entropy(logits.float().flatten(0, 1), tokens[:, 1:].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


def decode(model, tokens, prompt):
    """Logits after each token of (batch, L) from the prompt's last on, one token at a time."""
    logits, caches = model.prefill(tokens[:, :prompt].contiguous())
    out = [logits]
    pos = torch.full(tokens.shape[:1], prompt, dtype=torch.int32, device=tokens.device)
    for i in range(prompt, tokens.shape[1]):
        out.append(model.step(tokens[:, i].contiguous(), caches, pos))
        pos += 1
    return torch.stack(out, 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--tokens", type=int, default=64)
    a = ap.parse_args()
    torch.manual_seed(0)
    model = HybridModel().cuda()
    losses = train(model, sequence(8, 513, 256, "cuda"), a.steps)
    print(f"training: loss {losses[0]:.3f} -> {losses[-1]:.3f} in {len(losses)} steps", flush=True)
    tokens = sequence(4, a.prompt + a.tokens, 256, "cuda", seed=1)
    decode(model, tokens[:, :a.prompt + 2], a.prompt)
    torch.cuda.synchronize()
    begin = time.perf_counter()
    got = decode(model, tokens, a.prompt).float()
    torch.cuda.synchronize()
    took = time.perf_counter() - begin
    with torch.no_grad():
        want = model(tokens)[:, a.prompt - 1:].float()
    print(f"decoding: {a.prompt} tokens at once and {a.tokens} one by one, 4 sequences, in {took * 1e3:.1f} ms; "
          f"largest difference from the whole sequence's logits {float((got - want).abs().max()):.3f} "
          f"of {float(want.abs().max()):.1f}")


if __name__ == "__main__":
    main()
