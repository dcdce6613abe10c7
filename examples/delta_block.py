"""Blocks of a language model on the operators of libssm_delta: delta-rule
layers and sliding-window attention with normalised queries and keys in turn,
each after a residual addition with RMS norm, the attention's cache in 8 bits.

    python examples/delta_block.py [--steps 30] [--prompt 1000] [--tokens 64]

trains a small model on a synthetic sequence, reads a prompt in one pass, and
goes on token by token from the delta rule's states and the 8-bit caches,
comparing the tokens' outputs with those of the whole sequence.
"""
import argparse
import os
import sys
import time

import torch
from torch import nn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for path in (ROOT, os.path.join(ROOT, "examples")):
    if path not in sys.path:
        sys.path.insert(0, path)
import state_space_model_ssm_amd as ssm  # noqa: E402
from hybrid_block import BF16, AddNorm, Attention, decode, sequence, train  # noqa: E402


class DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, lengths):
        y, _, states = ssm.gdr_fwd(q, k, v, g, beta, lengths=lengths, return_h_last=False, return_states=True)
        ctx.save_for_backward(q, k, v, g, beta, states, lengths)
        return y

    @staticmethod
    def backward(ctx, dy):
        *args, states, lengths = ctx.saved_tensors
        return *ssm.gdr_bwd(*args, states, dy.contiguous(), lengths=lengths, return_dh0=False)[:5], None


class HeadNorms(torch.autograd.Function):
    """Norms of queries and keys by heads, and their rotation by position if there are frequencies."""

    @staticmethod
    def forward(ctx, q, k, wq, wk, inv_freq):
        ctx.save_for_backward(q, k, wq, wk, inv_freq)
        return ssm.qk_norm_fwd(q, k, wq, wk, inv_freq=inv_freq)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, wq, wk, inv_freq = ctx.saved_tensors
        learned = wq.requires_grad or wk.requires_grad
        return *ssm.qk_norm_bwd(q, k, wq, wk, dq.contiguous(), dk.contiguous(), inv_freq=inv_freq, return_dw=learned), None


class DeltaMixer(nn.Module):
    """Queries and keys of unit length; a decay and a writing strength per value head."""

    def __init__(self, dim, qk_heads, heads, kdim, vdim):
        super().__init__()
        self.split, self.dims = (2 * qk_heads * kdim, heads * vdim), (kdim, vdim)
        self.proj = nn.Linear(dim, sum(self.split), bias=False, dtype=BF16)
        self.gates = nn.Linear(dim, 2 * heads, bias=False, dtype=BF16)
        self.out = nn.Linear(heads * vdim, dim, bias=False, dtype=BF16)
        self.log_rate = nn.Parameter(torch.linspace(-4.0, 0.0, heads))   # slow and fast heads
        self.register_buffer("unit", torch.full((kdim,), kdim ** -0.5))  # a norm of 1, not of sqrt(kdim)

    def parts(self, x):
        qk, v = self.proj(x).split(self.split, -1)
        q, k = qk.unflatten(-1, (-1, self.dims[0])).chunk(2, -2)
        decay, beta = self.gates(x).float().chunk(2, -1)
        g = -torch.exp(self.log_rate) * nn.functional.softplus(decay)
        return q, k, v.unflatten(-1, (-1, self.dims[1])), g, torch.sigmoid(beta)

    def forward(self, x, lengths):
        q, k, v, g, beta = self.parts(x)
        q, k = HeadNorms.apply(q, k, self.unit, self.unit, None)
        return self.out(DeltaRule.apply(q, k, v, g, beta, lengths).flatten(-2))

    def prefill(self, x):
        q, k, v, g, beta = self.parts(x)
        y, state = ssm.gdr_fwd(*ssm.qk_norm_fwd(q, k, self.unit, self.unit), v, g, beta)
        return self.out(y.flatten(-2)), state

    def step(self, x, state, pos):
        q, k, v, g, beta = self.parts(x)
        y, _ = ssm.gdr_step(*ssm.qk_norm_fwd(q, k, self.unit, self.unit), v, g, beta, state)   # state: in place
        return self.out(y.flatten(-2))


class NormedWindowMixer(nn.Module):
    """Attention over a window and sinks, of normalised and rotated queries and keys; decoding holds them in 8 bits."""

    def __init__(self, dim, heads, kv_heads, headdim, window, sinks):
        super().__init__()
        self.split, self.headdim, self.window, self.sinks = (heads, kv_heads, kv_heads), headdim, window, sinks
        self.qkv = nn.Linear(dim, sum(self.split) * headdim, bias=False, dtype=BF16)
        self.out = nn.Linear(heads * headdim, dim, bias=False, dtype=BF16)
        self.wq, self.wk = (nn.Parameter(torch.ones(headdim)) for _ in range(2))
        self.register_buffer("inv_freq", 10000.0 ** -(torch.arange(headdim // 2) * 2.0 / headdim))

    def parts(self, x):
        return self.qkv(x).unflatten(-1, (-1, self.headdim)).split(self.split, -2)

    def forward(self, x, lengths):
        q, k, v = self.parts(x)
        q, k = HeadNorms.apply(q, k, self.wq, self.wk, self.inv_freq)
        return self.out(Attention.apply(q, k, v, self.window, self.sinks, lengths).flatten(-2))

    def prefill(self, x):
        q, k, v = self.parts(x)
        ssm.qk_norm_fwd(q, k, self.wq, self.wk, inv_freq=self.inv_freq, q_out=q, k_out=k)    # in their places
        y, _ = ssm.swa_fwd(q, k, v, window=self.window, sinks=self.sinks, return_lse=False)
        cache = ssm.swa_q8_cache(x.shape[0], self.split[1], self.window, self.headdim, sinks=self.sinks, device=x.device)
        ssm.swa_q8_fill(k, v, cache, sinks=self.sinks)
        return self.out(y.flatten(-2)), cache

    def step(self, x, cache, pos):
        q, k, v = self.parts(x)
        ssm.qk_norm_fwd(q, k, self.wq, self.wk, inv_freq=self.inv_freq, pos=pos, q_out=q, k_out=k)
        return self.out(ssm.swa_q8_step(q, k, v, cache, pos, sinks=self.sinks).flatten(-2))


class DeltaModel(nn.Module):
    """Tokens -> logits: `layers` pairs of a delta-rule and a window mixer."""

    def __init__(self, vocab=256, dim=512, layers=2, qk_heads=4, heads=8, kv_heads=2, headdim=64, window=256, sinks=4):
        super().__init__()
        self.embed = nn.Embedding(vocab, dim, dtype=BF16)
        self.mixers = nn.ModuleList()
        for _ in range(layers):
            self.mixers += [DeltaMixer(dim, qk_heads, heads, headdim, headdim),
                            NormedWindowMixer(dim, heads, kv_heads, headdim, window, sinks)]
        self.norms = nn.ParameterList(nn.Parameter(torch.ones(dim)) for _ in range(2 * layers + 1))
        self.head = nn.Linear(dim, vocab, bias=False, dtype=BF16)

    def forward(self, tokens, lengths=None):
        """Logits of (batch, L) tokens, of which each row has `lengths`."""
        x, s = self.embed(tokens), torch.zeros_like(self.embed.weight[:1]).expand(*tokens.shape, -1).contiguous()
        for norm, mixer in zip(self.norms, self.mixers):
            y, s = AddNorm.apply(x, s, norm)
            x = mixer(y, lengths)
        return self.head(AddNorm.apply(x, s, self.norms[-1])[0])

    @torch.no_grad()
    def prefill(self, tokens):
        """Logits of the prompt's last token, and the states and caches to go on from."""
        x, s, kept = self.embed(tokens), None, []
        for norm, mixer in zip(self.norms, self.mixers):
            y, s = ssm.rms_add_fwd(x, norm, s)
            x, one = mixer.prefill(y)
            kept.append(one)
        return self.head(ssm.rms_add_fwd(x[:, -1].contiguous(), self.norms[-1], s[:, -1].contiguous())[0]), kept

    @torch.no_grad()
    def step(self, token, kept, pos):
        """Logits after one token per row, (batch,), at positions pos (int32)."""
        x, s = self.embed(token), None
        for norm, mixer, one in zip(self.norms, self.mixers, kept):
            y, s = ssm.rms_add_fwd(x, norm, s)
            x = mixer.step(y, one, pos)
        return self.head(ssm.rms_add_fwd(x, self.norms[-1], s)[0])


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--tokens", type=int, default=64)
    a = ap.parse_args()
    torch.manual_seed(0)
    model = DeltaModel().cuda()
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
