"""A block of a hybrid model: a long convolution over the channels, then a
layer of the gated delta rule, trained on whole sequences and served token by
token: the rule from its state, the convolution from the tokens seen so far.

    python examples/hybrid_block.py [--train-steps 200] [--new-tokens 32]

The block runs the library's operators as a program would:
  FFTConv                     the long convolution of the training pass
  QKNorm                      unit-norm keys and queries, rotated by position
  GatedDelta.forward_train    the sequence, and what its gradients need
  GatedDelta.backward, QKNorm.backward, FFTConv.backward
  GatedDelta.forward          a prompt, packed with others, to its state
  GatedDelta.step, FFTConv    then one token at a time
It is trained to give what a second block with other random weights gives on
a synthetic batch.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fft_long_convolution_amd.delta import GatedDelta, QKNorm  # noqa: E402
from fft_long_convolution_amd.fftconv import FFTConv  # noqa: E402


class LongConv(torch.autograd.Function):
    """u [B, H, N], k [H, N] -> causal convolution."""

    @staticmethod
    def forward(ctx, u, k, conv):
        ctx.save_for_backward(u, k)
        ctx.conv = conv
        return conv.forward(u, conv.kernel_spectrum(k))

    @staticmethod
    def backward(ctx, dy):
        u, k = ctx.saved_tensors
        adjoint = ctx.conv.kernel_spectrum(k, kind="causal_adjoint")
        du, dk = ctx.conv.backward(u, dy.contiguous(), adjoint)
        return du, dk, None


class Norm(torch.autograd.Function):
    """Norms and rotation of q and k [B, T, H, D]."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin, positions, norm):
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, positions)
        ctx.norm = norm
        return norm.forward(q, k, q_weight, k_weight, cos, sin, positions)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, *rest = ctx.saved_tensors
        return (*ctx.norm.backward(q, k, dq, dk, *rest), None, None, None, None)


class Rule(torch.autograd.Function):
    """The gated delta rule over sequences."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, rule):
        o, _, saved = rule.forward_train(q, k, v, g, beta)
        ctx.save_for_backward(q, k, v, g, beta, saved)
        ctx.rule = rule
        return o

    @staticmethod
    def backward(ctx, do):
        *ins, saved = ctx.saved_tensors
        return (*ctx.rule.backward(*ins, do, saved)[:5], None)


class HybridBlock(torch.nn.Module):
    def __init__(self, width, heads, N, dtype="bf16"):
        super().__init__()
        self.width, self.heads, self.D = width, heads, width // heads
        D = self.D
        kind = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[dtype]
        self.conv = FFTConv(N, dtype=dtype)
        self.norm = QKNorm(D, rotary_dim=D // 2 // 16 * 16, norm="l2", dtype=dtype)
        self.rule = GatedDelta(D, D, dtype=dtype)
        self.kernel = torch.nn.Parameter(0.02 * torch.randn(width, N) *
                                         torch.exp(-torch.arange(N) / 64.0))
        self.qkv = torch.nn.Linear(width, 3 * width, bias=False).to(kind)
        self.gates = torch.nn.Linear(width, 2 * heads).to(kind)
        self.out = torch.nn.Linear(width, width, bias=False).to(kind)
        self.weights = torch.nn.Parameter(torch.ones(2, D))
        R = self.norm.rotary_dim
        turn = torch.arange(2 * N)[:, None] * 1e-4 ** (torch.arange(R // 2) / max(R // 2, 1))
        self.register_buffer("cos", turn.cos())
        self.register_buffer("sin", turn.sin())

    def mix(self, x):
        """The long convolution on top of x [B, N, width]."""
        return x + LongConv.apply(x.transpose(1, 2).contiguous(), self.kernel,
                                  self.conv).transpose(1, 2)

    def heads_of(self, x):
        """q, k, v [..., heads, D], log decays and write strengths of tokens."""
        q, k, v = (y.unflatten(-1, (self.heads, self.D))
                   for y in self.qkv(x).chunk(3, dim=-1))
        a, b = self.gates(x).float().chunk(2, dim=-1)
        return q, k, v, -0.01 * torch.nn.functional.softplus(a), torch.sigmoid(b)

    def rotated(self, q, k, positions):
        return Norm.apply(q, k, self.weights[0], self.weights[1], self.cos, self.sin, positions,
                          self.norm)

    def forward(self, x):
        """Training: x [B, N, width] through both mixers."""
        x = self.mix(x)
        q, k, v, g, beta = self.heads_of(x)
        positions = torch.arange(x.shape[1], device=x.device).expand(x.shape[:2]).contiguous()
        q, k = self.rotated(q, k, positions)
        return self.out(Rule.apply(q, k, v, g, beta, self.rule).flatten(2))

    @torch.no_grad()
    def prefill(self, x, bounds):
        """Prompts packed in one row x [1, T, width], bounds int64 [n + 1]:
        outputs, and of each its tokens [n, N, width] and its state."""
        lengths = bounds.diff()
        row = torch.repeat_interleave(torch.arange(len(lengths), device=x.device), lengths)
        position = torch.arange(x.shape[1], device=x.device) - bounds[row]
        seen = x.new_zeros(len(lengths), self.conv.N, self.width)
        seen[row, position] = x[0]
        q, k, v, g, beta = self.heads_of(self.mix(seen)[row, position][None])
        q, k = self.rotated(q, k, position[None])
        o, state = self.rule.forward(q, k, v, g, beta, cu_seqlens=bounds)
        return self.out(o.flatten(2)), seen, state

    @torch.no_grad()
    def decode(self, x, seen, state, slots, positions):
        """The next token x [n, width] of each request, whose earlier ones are
        seen[slot] and whose state is state[slot]; both take it in.  The
        convolution is causal, so what stands behind the token does not
        matter; it is taken over the whole length here."""
        seen[slots, positions] = x
        rows = torch.arange(len(slots), device=x.device)
        q, k, v, g, beta = self.heads_of(self.mix(seen[slots])[rows, positions])
        q, k = self.rotated(q[:, None], k[:, None], positions[:, None])
        o = self.rule.step(q[:, 0], k[:, 0], v, g, beta, state, slots=slots)
        return self.out(o.flatten(1))


def serve(block, x, lengths, new_tokens):
    """Prompts x[b, :lengths[b]], then new_tokens of each one at a time:
    pairs of what serving and what the training pass over the whole x gives."""
    whole = block(x)
    bounds = torch.tensor([0, *lengths], device=x.device).cumsum(0)
    y, seen, state = block.prefill(torch.cat([x[b, :n] for b, n in enumerate(lengths)])[None],
                                   bounds)
    pairs = [(y[0, bounds[b]:bounds[b + 1]], whole[b, :n]) for b, n in enumerate(lengths)]
    # requests live in pools, among others
    slots = torch.arange(len(lengths), device=x.device) * 3 + 2
    seen_pool = seen.new_zeros(3 * len(lengths) + 2, *seen.shape[1:])
    state_pool = state.new_zeros(3 * len(lengths) + 2, *state.shape[1:])
    seen_pool[slots], state_pool[slots] = seen, state
    at = torch.tensor(lengths, device=x.device)
    rows = torch.arange(len(lengths), device=x.device)
    for _ in range(new_tokens):
        y = block.decode(x[rows, at], seen_pool, state_pool, slots, at)
        pairs.append((y, whole[rows, at]))
        at = at + 1
    return pairs


def worst_error(pairs):
    """The largest error of a pair, relative to the norm of the same tokens."""
    return max(((y - w).float().norm() / w.float().norm()).item() for y, w in pairs)


def main(width=128, heads=2, N=256, batch=4, train_steps=200, new_tokens=32, log=print):
    torch.manual_seed(0)
    block, other = HybridBlock(width, heads, N).cuda(), HybridBlock(width, heads, N).cuda()
    kind = block.qkv.weight.dtype
    opt = torch.optim.Adam(block.parameters(), lr=3e-3)
    x = torch.randn(batch, N, width, device="cuda").to(kind)
    with torch.no_grad():
        want = other(x).float()
    losses = []
    for i in range(train_steps):
        y = block(x)
        loss = ((y.float() - want) ** 2).mean() / want.square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
        if i % 20 == 0 or i + 1 == train_steps:
            log("step %d  loss %.4f" % (i, losses[-1]))

    # serving: two prompts of different lengths, then token by token, must
    # give what the training pass gives over the whole sequences
    with torch.no_grad():
        x = torch.randn(2, N, width, device="cuda").to(kind)
        error = worst_error(serve(block, x, (N - new_tokens, N - new_tokens - 37), new_tokens))
    log("prefill and %d decoded tokens against the training pass: %.2e" % (new_tokens, error))
    return losses, error


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--width", type=int, default=128)
    parser.add_argument("--heads", type=int, default=2)
    parser.add_argument("--length", type=int, default=256, help="a power of two, 256 or more")
    parser.add_argument("--train-steps", type=int, default=200)
    parser.add_argument("--new-tokens", type=int, default=32)
    a = parser.parse_args()
    main(a.width, a.heads, a.length, train_steps=a.train_steps, new_tokens=a.new_tokens)
