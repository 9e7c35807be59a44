"""A residual recurrent block from this library's operators, trained over whole (or packed) sequences
and served token by token.

    norm -> one projection to (x, r, i, z) -> gated recurrence (and, in a bidirectional block, a second
    one from the sequence's end) -> gated norm -> projection -> scaled residual + next block's norm

The recurrence, the gated norm and the junction between two blocks (post-norm, residual scale,
pre-norm) are the library's kernels; the projections are plain matrix products. Run

    python -m bidirectional_selective_scan_amd.recurrent_block

on a GPU to train a small stack on a running-mean task and decode with it token by token.
"""
from __future__ import annotations

import math

import torch
from torch import nn

from . import binding
from .autograd import block_norm, gated_recurrence


class RecurrentBlock(nn.Module):
    """One block of width d with d_inner recurrence channels. ``bidirectional`` adds a recurrence from
    the end of every sequence (then it cannot be served token by token)."""

    def __init__(self, d: int, d_inner: int, bidirectional: bool = False, c: float = 8.0, dtype=torch.bfloat16):
        super().__init__()
        self.c, self.d_inner, self.directions = c, d_inner, 2 if bidirectional else 1
        self.wide = d_inner * (3 * self.directions + 1)
        self.w_in = nn.Parameter((torch.randn(d, self.wide) / math.sqrt(d)).to(dtype))
        self.w_out = nn.Parameter((torch.randn(d_inner, d) / math.sqrt(d_inner)).to(dtype))
        a = torch.rand(self.directions, d_inner) * 0.099 + 0.9          # slowest decay of a channel
        self.lam = nn.Parameter(torch.log(torch.expm1(-torch.log(a) / c)))
        self.w_gated = nn.Parameter(torch.ones(d_inner))                # norm of the gated recurrence
        self.w_post = nn.Parameter(torch.ones(d))                       # norm of the block's output
        self.gamma = nn.Parameter(torch.full((d,), 0.5))                # residual scale
        self.w_next = nn.Parameter(torch.ones(d))                       # norm in front of the next block

    def _split(self, n):
        parts = (n @ self.w_in).split(self.d_inner, dim=-1)             # slices of one array
        return parts[:-1], parts[-1]

    def forward(self, n, residual, offsets=None):
        """n: the block's normed input (B, L, d); residual: the fp32 residual stream. Returns the next
        block's (n, residual)."""
        xri, z = self._split(n)
        y = None
        for k in range(self.directions):
            h, _ = gated_recurrence(*xri[3 * k:3 * k + 3], self.lam[k], self.c, offsets=offsets, reverse=k == 1)
            y = h if y is None else y + h
        g, _ = block_norm(y, z, self.w_gated)
        residual, n = block_norm(g @ self.w_out, None, self.w_post, residual, self.gamma, self.w_next)
        return n, residual

    @torch.no_grad()
    def prefill(self, n, residual):
        """``forward`` that also returns the state after the last token of every sequence (B, d_inner)."""
        if self.directions != 1:
            raise ValueError("a bidirectional block has no state to go on from")
        xri, z = self._split(n)
        y, state = binding.gated_fwd(*xri, self.lam[0], self.c)
        g, _ = binding.block_norm(y, z, self.w_gated)
        residual, n = binding.block_norm(g @ self.w_out, None, self.w_post, residual, self.gamma, self.w_next)
        return n, residual, state

    @torch.no_grad()
    def step(self, n, residual, state):
        """One token of every stream: n, residual (B, d), state (B, d_inner) updated in place."""
        xri, z = self._split(n)
        y = binding.gated_step(*xri, self.lam[0], state, self.c)
        g, _ = binding.block_norm(y, z, self.w_gated)
        residual, n = binding.block_norm(g @ self.w_out, None, self.w_post, residual, self.gamma, self.w_next)
        return n, residual


class RecurrentStack(nn.Module):
    """Blocks between an input and an output projection; the residual stream is fp32."""

    def __init__(self, d_in: int, d: int, d_inner: int, d_out: int, depth: int, bidirectional: bool = False,
                 dtype=torch.bfloat16):
        super().__init__()
        self.dtype = dtype
        self.w_in = nn.Parameter(torch.randn(d_in, d) / math.sqrt(d_in))
        self.w_first = nn.Parameter(torch.ones(d))
        self.blocks = nn.ModuleList(RecurrentBlock(d, d_inner, bidirectional, dtype=dtype) for _ in range(depth))
        self.w_head = nn.Parameter((torch.randn(d, d_out) / math.sqrt(d)).to(dtype))

    def _embed(self, u):
        residual = (u.float() @ self.w_in).contiguous()
        _, n = block_norm(residual.to(self.dtype), w_pre=self.w_first)
        return n, residual

    def forward(self, u, offsets=None):
        n, residual = self._embed(u)
        for b in self.blocks:
            n, residual = b(n, residual, offsets)
        return (n @ self.w_head).float()

    @torch.no_grad()
    def prefill(self, u):
        n, residual = self._embed(u)
        states = []
        for b in self.blocks:
            n, residual, s = b.prefill(n, residual)
            states.append(s)
        return (n @ self.w_head).float(), states

    @torch.no_grad()
    def step(self, u, states):
        n, residual = self._embed(u)
        for b, s in zip(self.blocks, states):
            n, residual = b.step(n, residual, s)
        return (n @ self.w_head).float()


def running_mean_batch(batch, length, d_in, generator, device="cuda:0"):
    """Inputs u ~ N(0, 1) and their exponential running mean of rate 0.95 (the task to learn)."""
    u = torch.randn(batch, length, d_in, generator=generator, device=device)
    w = 0.95 ** torch.arange(length, device=device, dtype=torch.float32)
    kernel = torch.tril(w[(torch.arange(length, device=device)[:, None] - torch.arange(length, device=device)).clamp(min=0)])
    return u, torch.einsum("ts,bsd->btd", kernel, u) * 0.3


def main(steps: int = 60, device: str = "cuda:0"):
    """Trains a small stack for ``steps`` steps, then decodes a prompt's continuation token by token.
    Returns (first loss, last loss, largest difference between decoding and the whole sequence)."""
    torch.manual_seed(0)
    gen = torch.Generator(device=device)
    gen.manual_seed(0)
    model = RecurrentStack(8, 128, 192, 8, depth=2).to(device)
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        u, want = running_mean_batch(16, 197, 8, gen, device)
        loss = torch.nn.functional.mse_loss(model(u), want)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    u, _ = running_mean_batch(4, 80, 8, gen, device)
    with torch.no_grad():
        whole = model(u)
    _, states = model.prefill(u[:, :50])
    out = torch.stack([model.step(u[:, t], states) for t in range(50, 80)], 1)
    diff = (out - whole[:, 50:]).abs().max().item()
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps; decoding differs from the whole sequence by {diff:.3e}")
    return losses[0], losses[-1], diff


if __name__ == "__main__":
    main()
