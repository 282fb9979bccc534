"""A deep stack of gated linear recurrences over packed sequences: trained, then run frame by frame.

Each layer reads the normalised residual stream, projects it to the gates i, f, z and an output gate o (the library's
input projection over all frames at once), scans h_t = sig(f) h_{t-1} + sig(i) z over every sequence, and adds its
normalised, gated and scaled output back to the stream; the same call forms the next layer's normalised input.  After a
few steps of gradient descent the same weights run as a streaming recogniser would run them: one frame of every stream at
a time, states in a cache of slots, idle streams left alone.

    python examples/gated_recurrence.py
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from padding_free_variable_gb300 import ops  # noqa: E402

PARAMS = ("w_post", "scale", "w_pre")


class GatedRecurrenceStack:
    """`layers` layers of `width` units over one packed batch (fp32); buffers made once, kept from step to step."""

    def __init__(self, plan: ops.Plan, width: int, layers: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        H, n, dev = width, plan.rows, "cuda"
        self.plan, self.H, self.L = plan, H, layers

        def new(*shape):
            return torch.empty(shape, device=dev)

        def normal(*shape, std):
            return torch.randn(shape, generator=g, device=dev) * std

        # per layer the projection's weights [4H, H], rows i, f, z, o, with the forget gates biased towards keeping, and
        # the norms around the layer: w_post and scale behind it, w_pre in front of the next one (the last layer's: the head)
        self.W = [normal(4 * H, H, std=H ** -0.5) for _ in range(layers)]
        self.b = [torch.cat([torch.zeros(H), torch.full((H,), 2.0), torch.zeros(2 * H)]).to(dev) for _ in range(layers)]
        self.first = torch.ones(H, device=dev)
        self.norm = [{"w_post": torch.ones(H, device=dev), "scale": torch.full((H,), 0.5, device=dev),
                      "w_pre": torch.ones(H, device=dev)} for _ in range(layers)]
        self.glr = ops.glr_shape(H, 1, False, "gated")
        self.pre = ops.block_norm_shape(H, "rms", "none", post_kind="none")
        self.block = ops.block_norm_shape(H, "rms", "silu")
        self.proj_shape = ops.layer_shape(H, H, 1, False)
        # the LSTM-shaped parts of the projection's call that a layer without recurrent weights does not have
        self.unused = {"R": torch.zeros(4 * H, H, device=dev), "peep": torch.zeros(3, H, device=dev)}
        self.x = [new(n, H) for _ in range(layers + 1)]                 # the residual stream
        self.n = [new(n, H) for _ in range(layers + 1)]                 # what each layer (and the head) reads
        self.gates = [new(n, 4 * H) for _ in range(layers)]
        self.y = [new(n, 1, H) for _ in range(layers)]
        self.h_n = [new(1, plan.batch, H) for _ in range(layers)]
        self.ws = [torch.empty(ops.glr_workspace_bytes(plan, self.glr), dtype=torch.uint8, device=dev) for _ in range(layers)]
        self.first_stats, self.stats = new(n, 4), [new(n, 4) for _ in range(layers)]
        self.scratch = torch.empty(max(ops.block_norm_scratch_bytes(s, n) for s in (self.pre, self.block)), dtype=torch.uint8,
                                   device=dev)

    def views(self, t):
        """The i, f, z blocks [rows, 1, H] and the o block [rows, H] of a projection's rows."""
        v = t.view(t.shape[0], 1, 4, self.H)
        return v[:, :, 0], v[:, :, 1], v[:, :, 2], t[:, 3 * self.H:]

    def forward(self, x):
        """x [rows, H] packed; returns the head's input."""
        self.x[0].copy_(x)
        ops.block_norm_forward(self.pre, self.x[0], None, None, {"w_pre": self.first}, None, self.n[0], self.first_stats)
        for k in range(self.L):
            ops.input_projection(self.plan, self.proj_shape, {"W": self.W[k], "b": self.b[k], **self.unused}, self.n[k],
                                 self.gates[k])
            i, f, z, o = self.views(self.gates[k])
            ops.glr_forward(self.plan, self.glr, f, z, i, None, self.y[k], self.h_n[k], self.ws[k])
            ops.block_norm_forward(self.block, self.x[k], self.y[k][:, 0], o, self.norm[k], self.x[k + 1], self.n[k + 1],
                                   self.stats[k])
        return self.n[-1]

    def backward(self, dn):
        """dL/d(head's input) -> gradients of every weight, in the order of `parameters`."""
        grads, dx = [], None
        for k in reversed(range(self.L)):
            i, f, z, o = self.views(self.gates[k])
            dgates = torch.empty_like(self.gates[k])
            di, df, dz, do = self.views(dgates)
            dy, dxk = torch.empty_like(self.y[k]), torch.empty_like(self.x[k])
            dp = {p: torch.empty_like(self.first) for p in PARAMS}
            ops.block_norm_backward(self.block, self.x[k], self.y[k][:, 0], o, self.norm[k], self.stats[k], dx, dn, dxk,
                                    dy[:, 0], do, dp, self.scratch)
            ops.glr_backward(self.plan, self.glr, f, z, i, self.ws[k], dy, None, df, dz, di, None)
            grads += [dp[p] for p in reversed(PARAMS)] + [dgates.sum(0), dgates.t() @ self.n[k]]
            dn, dx = dgates @ self.W[k], dxk
        out, dfirst = torch.empty_like(self.x[0]), {"w_pre": torch.empty_like(self.first)}
        ops.block_norm_backward(self.pre, self.x[0], None, None, {"w_pre": self.first}, self.first_stats, dx, dn, out, None, None,
                                dfirst, self.scratch)
        return [dfirst["w_pre"]] + grads[::-1]

    def parameters(self):
        out = [self.first]
        for k in range(self.L):
            out += [self.W[k], self.b[k]] + [self.norm[k][p] for p in PARAMS]
        return out

    def stream(self, slots: int):
        """State caches of `slots` streams, one a layer, and the function that takes their next frames."""
        cache = [torch.zeros(slots, self.H, device="cuda") for _ in range(self.L)]

        def step(frames, at):
            """frames [streams, H], at [streams] int32: each one's slot (-1: idle, its output means nothing)."""
            m = frames.shape[0]
            x, n, y = frames, torch.empty_like(frames), torch.empty(m, 1, self.H, device="cuda")
            ops.block_norm_forward(self.pre, x, None, None, {"w_pre": self.first}, None, n)
            for k in range(self.L):
                gates = torch.nn.functional.linear(n, self.W[k], self.b[k])
                i, f, z, o = self.views(gates)
                ops.glr_step(self.glr, f, z, i, cache[k], cache[k], y, at)
                x1, n = torch.empty_like(x), torch.empty_like(x)
                ops.block_norm_forward(self.block, x, y[:, 0], o, self.norm[k], x1, n)
                x = x1
            return n

        return step


def train(lengths, width=64, layers=2, steps=30, rate=0.3, seed=0):
    """Gradient descent on recalling a mean of the past; returns the stack and the losses."""
    plan = ops.Plan(lengths)
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.normal(size=(plan.frames, width)).astype(np.float32)).cuda()
    # target: an exponential mean of a few fixed mixtures of the frames so far, sequence by sequence
    mix = torch.from_numpy(rng.normal(size=(width, 8)).astype(np.float32)).cuda() * width ** -0.5
    want, at = torch.empty(plan.frames, 8, device="cuda"), 0
    for n in lengths:
        m = torch.zeros(8, device="cuda")
        for t in range(at, at + n):
            m = 0.9 * m + 0.3 * (x[t] @ mix)
            want[t] = m
        at += n
    xp, wp = plan.pack(x), plan.pack(want)
    stack = GatedRecurrenceStack(plan, width, layers, seed)
    head = torch.zeros(width, 8, device="cuda")
    losses = []
    for _ in range(steps):
        n = stack.forward(xp)
        err = n @ head - wp
        losses.append(float(err.square().mean()))
        d = err * (2.0 / err.numel())
        grads = stack.backward(d @ head.t())
        head -= rate * (n.t() @ d)
        for p, g in zip(stack.parameters(), grads):
            p -= rate * g
    return stack, xp, losses


def compare_streaming(stack, xp, lengths):
    """The scan's outputs against the same frames taken one at a time from every stream; the largest difference."""
    whole = stack.plan.unpack(stack.forward(xp))
    x = stack.plan.unpack(xp)
    starts = np.concatenate([[0], np.cumsum(lengths)])
    step = stack.stream(len(lengths) + 3)
    slots = np.arange(len(lengths))[::-1] + 2           # anywhere in the cache
    worst = 0.0
    for t in range(max(lengths)):
        on = np.array([t < n for n in lengths])
        rows = torch.from_numpy(np.where(on, starts[:-1] + t, 0)).cuda()
        at = torch.from_numpy(np.where(on, slots, -1).astype(np.int32)).cuda()
        out = step(x[rows], at)
        on = torch.from_numpy(on).cuda()
        worst = max(worst, float((out - whole[rows])[on].abs().max()))
    return worst


def main():
    lengths = [70, 33, 5, 128, 64, 1, 97]
    stack, xp, losses = train(lengths)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps over {stack.plan.frames} frames")
    print(f"frame by frame against the scan: largest difference {compare_streaming(stack, xp, lengths):.2e}")


if __name__ == "__main__":
    main()
