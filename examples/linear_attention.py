"""A deep stack of linear attention layers over packed sequences: trained, then run frame by frame.

Each layer reads the normalised residual stream, projects it to queries, keys, values and an output gate (the library's input
projection over all frames at once), normalises and rotates each head's query and key by its frame's position, lets every
head attend to its sequence's past with a decay of its own, and adds its normalised, gated and scaled output back to the
stream; the same call forms the next layer's normalised input.  Afterwards the same weights run as a streaming recogniser would
run them: one frame of every stream at a time, states in a cache of slots, idle streams left alone.

    python examples/linear_attention.py
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from padding_free_variable_gb300 import ops  # noqa: E402

PARAMS = ("w_post", "scale", "w_pre")


class LinearAttentionStack:
    """`layers` layers of `heads` heads of `size` values over one packed batch (fp32); buffers kept from step to step."""

    def __init__(self, plan: ops.Plan, heads: int, size: int, layers: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        W, n, dev = heads * size, plan.rows, "cuda"
        self.plan, self.heads, self.size, self.W, self.L = plan, heads, size, W, layers

        def new(*shape):
            return torch.empty(shape, device=dev)

        # per layer the projection's weights [4W, W], rows q, k, v, gate; the heads' norms; the norms around the layer
        self.P = [torch.randn(4 * W, W, generator=g, device=dev) * W ** -0.5 for _ in range(layers)]
        self.b = [torch.zeros(4 * W, device=dev) for _ in range(layers)]
        self.wq, self.wk = ([torch.ones(size, device=dev) for _ in range(layers)] for _ in range(2))
        self.first = torch.ones(W, device=dev)
        self.norm = [{"w_post": torch.ones(W, device=dev), "scale": torch.full((W,), 0.5, device=dev), "w_pre": torch.ones(W, device=dev)}
                     for _ in range(layers)]
        # memories from a few frames to a few hundred; rotations of half of each head
        self.log_decay = torch.log1p(-2.0 ** -(2.0 + 6.0 * torch.arange(heads, device=dev) / heads))[None]
        self.turn = ops.qk_norm_shape(heads, heads, size, "rms", size // 2, "half")
        self.table = ops.rotary_table(ops.rotary_frequencies(size // 2))
        self.la = ops.la_shape(heads, size, size)
        self.pre = ops.block_norm_shape(W, "rms", "none", post_kind="none")
        self.block = ops.block_norm_shape(W, "rms", "silu")
        self.proj = ops.layer_shape(W, W, 1, False)
        # the LSTM-shaped parts of the projection's call that a layer without recurrent weights does not have
        self.unused = {"R": torch.zeros(4 * W, W, device=dev), "peep": torch.zeros(3, W, device=dev)}
        self.x, self.n = [new(n, W) for _ in range(layers + 1)], [new(n, W) for _ in range(layers + 1)]
        self.rows = [new(n, 4 * W) for _ in range(layers)]
        self.turned = [new(n, 2, heads, size) for _ in range(layers)]
        self.y = [new(n, 1, heads, size) for _ in range(layers)]
        self.first_stats, self.stats = new(n, 4), [new(n, 4) for _ in range(layers)]
        self.scratch = torch.empty(max(ops.block_norm_scratch_bytes(s, n) for s in (self.pre, self.block)) +
                                   ops.qk_norm_scratch_bytes(self.turn, n), dtype=torch.uint8, device=dev)

    def views(self, t):
        """q, k, v [rows, heads, size] and the gate [rows, W] of a projection's rows."""
        v = t.view(t.shape[0], 4, self.heads, self.size)
        return v[:, 0], v[:, 1], v[:, 2], t[:, 3 * self.W:]

    def forward(self, x):
        """x [rows, W] packed; returns the head's input."""
        self.x[0].copy_(x)
        ops.block_norm_forward(self.pre, self.x[0], None, None, {"w_pre": self.first}, None, self.n[0], self.first_stats)
        for i in range(self.L):
            ops.input_projection(self.plan, self.proj, {"W": self.P[i], "b": self.b[i], **self.unused}, self.n[i], self.rows[i])
            q, k, v, gate = self.views(self.rows[i])
            tq, tk = self.turned[i][:, 0], self.turned[i][:, 1]
            ops.qk_norm_forward(self.turn, q, k, self.wq[i], self.wk[i], self.table, None, tq, tk, plan=self.plan)
            ops.la_forward(self.plan, self.la, tq[:, None], tk[:, None], v[:, None], self.log_decay, None, self.y[i], None)
            ops.block_norm_forward(self.block, self.x[i], self.y[i].view(-1, self.W), gate, self.norm[i], self.x[i + 1],
                                   self.n[i + 1], self.stats[i])
        return self.n[-1]

    def backward(self, dn):
        """dL/d(head's input) -> gradients of every weight, in the order of `parameters`."""
        grads, dx = [], None
        for i in reversed(range(self.L)):
            q, k, v, gate = self.views(self.rows[i])
            drows = torch.empty_like(self.rows[i])
            dq, dk, dv, dgate = self.views(drows)
            tq, tk = self.turned[i][:, 0], self.turned[i][:, 1]
            dy, dxi = torch.empty_like(self.y[i]), torch.empty_like(self.x[i])
            dp = {p: torch.empty_like(self.first) for p in PARAMS}
            ops.block_norm_backward(self.block, self.x[i], self.y[i].view(-1, self.W), gate, self.norm[i], self.stats[i], dx, dn, dxi,
                                    dy.view(-1, self.W), dgate, dp, self.scratch)
            ops.la_backward(self.plan, self.la, tq[:, None], tk[:, None], v[:, None], self.log_decay, None, dy, None, dq[:, None],
                            dk[:, None], dv[:, None], None)
            dwq, dwk = torch.empty_like(self.wq[i]), torch.empty_like(self.wk[i])
            ops.qk_norm_backward(self.turn, q, k, self.wq[i], self.wk[i], self.table, None, dq, dk, dq, dk, dwq, dwk, self.scratch,
                                 plan=self.plan)
            grads += [dp[p] for p in reversed(PARAMS)] + [dwk, dwq, drows.sum(0), drows.t() @ self.n[i]]
            dn, dx = drows @ self.P[i], dxi
        out, dfirst = torch.empty_like(self.x[0]), {"w_pre": torch.empty_like(self.first)}
        ops.block_norm_backward(self.pre, self.x[0], None, None, {"w_pre": self.first}, self.first_stats, dx, dn, out, None, None,
                                dfirst, self.scratch)
        return [dfirst["w_pre"]] + grads[::-1]

    def parameters(self):
        out = [self.first]
        for i in range(self.L):
            out += [self.P[i], self.b[i], self.wq[i], self.wk[i]] + [self.norm[i][p] for p in PARAMS]
        return out

    def stream(self, slots: int):
        """State caches of `slots` streams, one a layer, and the function that takes their next frames."""
        cache = [torch.zeros(slots, self.heads, self.size, self.size, device="cuda") for _ in range(self.L)]

        def step(frames, at, positions):
            """frames [streams, W], at [streams] int32: each one's slot (-1: idle), positions [streams] int32."""
            m = frames.shape[0]
            x, n, y = frames, torch.empty_like(frames), torch.empty(m, 1, self.heads, self.size, device="cuda")
            ops.block_norm_forward(self.pre, x, None, None, {"w_pre": self.first}, None, n)
            for i in range(self.L):
                q, k, v, gate = self.views(torch.nn.functional.linear(n, self.P[i], self.b[i]))
                ops.qk_norm_forward(self.turn, q, k, self.wq[i], self.wk[i], self.table, positions, q, k)
                ops.la_step(self.la, q[:, None], k[:, None], v[:, None], self.log_decay, cache[i], cache[i], y, at)
                x1, n = torch.empty_like(x), torch.empty_like(x)
                ops.block_norm_forward(self.block, x, y.view(-1, self.W), gate, self.norm[i], x1, n)
                x = x1
            return n

        return step


def train(lengths, heads=4, size=16, layers=2, steps=30, rate=0.3, seed=0):
    """Gradient descent on recalling a mean of the past; returns the stack, its input and the losses."""
    plan, width = ops.Plan(lengths), heads * size
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.normal(size=(plan.frames, width)).astype(np.float32)).cuda()
    mix = torch.from_numpy(rng.normal(size=(width, 8)).astype(np.float32)).cuda() * width ** -0.5
    want, at = torch.empty(plan.frames, 8, device="cuda"), 0
    for n in lengths:
        m = torch.zeros(8, device="cuda")
        for t in range(at, at + n):
            m = 0.9 * m + 0.3 * (x[t] @ mix)
            want[t] = m
        at += n
    xp, wp = plan.pack(x), plan.pack(want)
    stack = LinearAttentionStack(plan, heads, size, layers, seed)
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
    """The whole sequences' outputs against the same frames taken one at a time from every stream; the largest difference."""
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
        out = step(x[rows], at, torch.full((len(lengths),), t, dtype=torch.int32, device="cuda"))
        on = torch.from_numpy(on).cuda()
        worst = max(worst, float((out - whole[rows])[on].abs().max()))
    return worst


def main():
    lengths = [70, 33, 5, 128, 64, 1, 97]
    stack, xp, losses = train(lengths)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps over {stack.plan.frames} frames")
    print(f"frame by frame against whole sequences: largest difference {compare_streaming(stack, xp, lengths):.2e}")


if __name__ == "__main__":
    main()
