"""A residual feed-forward network trained under emulated ZeRO-3 with the package's operators.

Layer l of the residual stream y (a row a token):

    z = Norm(y; pre_l)                         a = gelu(z W1 + b1)
    h = a W2 + b2                              y' = y + s * gate_l * Norm(h; post_l)

Its matrices and biases are one unit of a stage-3 plan: gathered from the ranks' shards before
they are used, and the ranks' 16-bit gradients are written by the backward pass straight into the
contributions that ``zero_step`` reduces.  The norms' gains and the gates are a few thousand
numbers, replicated, and stepped by ``zero_adamw`` with 8-bit moments, in one with the matrices: a
gradient that is not finite leaves out both, and one norm clips both.  ``zero_block_norm`` joins a
layer's end with the next one's start.

    python -m zero_sharded_mixed_03_gb300.feed_forward

trains a small one on a synthetic regression and prints the loss.
"""
from __future__ import annotations

from typing import Dict, List

import torch

from . import (ZERO_ACT_GELU, ZERO_ACT_NONE, ZERO_BF16, ZERO_FP32, ZERO_NORM_POST, ZERO_NORM_PRE,
               ZERO_NORM_RMS, ZERO_WEIGHT_IN_OUT, hyper, zero_adamw_bind, zero_adamw_check,
               zero_adamw_create, zero_adamw_destroy, zero_adamw_info, zero_adamw_step_with, zero_block_norm,
               zero_block_norm_backward, zero_block_norm_t, zero_block_norm_workspace, zero_linear,
               zero_linear_backward, zero_linear_t, zero_linear_workspace)
from .emulate import EmulatedGroup


class ShardedFeedForward:
    def __init__(self, layers: int, dim: int, inner: int, n_d: int, rows: int, residual_scale: float = 1.0,
                 eps: float = 1e-5, seed: int = 0):
        """rows: tokens of each rank's micro-batch."""
        self.layers, self.dim, self.inner, self.n_d, self.rows = layers, dim, inner, n_d, rows
        self.scale, self.eps = residual_scale, eps
        tensors = [dim * inner, inner, inner * dim, dim]                  # W1, b1, W2, b2
        self.at = [sum(tensors[:i]) for i in range(4)]
        self.group = EmulatedGroup(tensors * layers, n_d, 3, unit_first=[4 * u for u in range(layers)])
        gen = torch.Generator().manual_seed(seed)
        for u in range(layers):
            w = [torch.randn(n, generator=gen) * std for n, std in
                 zip(tensors, (dim ** -0.5, 0.0, inner ** -0.5, 0.0))]
            self._place(u, torch.cat(w))

        def new(*shape):
            return torch.empty(*shape, dtype=torch.bfloat16, device="cuda")

        # per layer, replicated: pre gain, post gain, gate; fp32 and the 16 bits that the kernels read
        self.vectors = torch.ones(layers, 3, dim, device="cuda")
        self.vectors16 = self.vectors.to(torch.bfloat16)
        self.vector_grads = torch.zeros(layers, 3, dim, device="cuda")
        self.rank_vector_grads = new(n_d, layers, 3, dim).zero_()
        self.opt = zero_adamw_create([dim] * (3 * layers), 8, ZERO_BF16, ZERO_FP32)
        info = zero_adamw_info(self.opt)
        self.moments = [torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")
                        for n in (info.moment_bytes, info.moment_bytes, info.scale_bytes, info.workspace_bytes)]
        ptrs = [[t.data_ptr() + i * dim * t.element_size() for i in range(3 * layers)]
                for t in (self.vectors, self.vectors16, self.vector_grads)]
        zero_adamw_bind(self.opt, *ptrs, *(t.data_ptr() for t in self.moments), 0, self._stream())
        # gathered units (two buffers in turn, on the one stream: nothing overlaps), activations of one
        # rank's micro-batch, contributions of every rank and unit
        self.full = [new(int(self.group.info.max_unit_pad)) for _ in range(2)]
        self.contribs = [[new(unit[3]).zero_() for _ in range(n_d)] for unit in self.group.units]
        self.y = [new(rows, dim) for _ in range(layers + 1)]
        self.z, self.h = ([new(rows, dim) for _ in range(layers)] for _ in range(2))
        self.pre, self.act = ([new(rows, inner) for _ in range(layers)] for _ in range(2))
        self.dy, self.dz, self.dh, self.da = new(rows, dim), new(rows, dim), new(rows, dim), new(rows, inner)
        self.workspace = torch.empty(16, dtype=torch.uint8, device="cuda")

    def close(self) -> None:
        self.group.close()
        if self.opt:
            zero_adamw_destroy(self.opt)
            self.opt = 0

    # ------------------------------------------------------------------ pieces

    @staticmethod
    def _stream() -> int:
        return torch.cuda.current_stream().cuda_stream

    def _place(self, unit: int, values: torch.Tensor) -> None:
        """A unit's initial parameters into the ranks' shards: 16 bits, and widened as the master."""
        padded = torch.zeros(self.group.units[unit][3], dtype=torch.bfloat16)
        padded[:values.numel()] = values.to(torch.bfloat16)
        for r in self.group.bound:
            _, off, n, _, size = self.group.shard_slices(r)[unit]
            part = padded[r * size:r * size + n].cuda()
            self.group.shard16[r][off:off + n] = part.view(torch.int16)
            self.group.state[r]["master"][0][off:off + n] = part.float()

    def unit16(self, unit: int) -> torch.Tensor:
        """The unit's gathered parameters, in one of two buffers."""
        dst = self.full[unit % 2]
        self.group.gather(unit, dst)
        return dst

    def _room(self, n: int) -> int:
        if self.workspace.numel() < n:
            self.workspace = torch.empty(n, dtype=torch.uint8, device="cuda")
        return self.workspace.data_ptr()

    def _linear(self, unit: torch.Tensor, layer: int, second: bool, **buffers) -> zero_linear_t:
        w, b = self.at[2:] if second else self.at[:2]
        sizes = (self.inner, self.dim) if second else (self.dim, self.inner)
        base = unit.data_ptr()
        return zero_linear_t(rows=self.rows, in_features=sizes[0], out_features=sizes[1], dtype16=ZERO_BF16,
                             layout=ZERO_WEIGHT_IN_OUT, activation=ZERO_ACT_NONE if second else ZERO_ACT_GELU,
                             w=base + 2 * w, bias=base + 2 * b, **buffers)

    def _vector(self, buf: torch.Tensor, layer: int, which: int) -> int:
        return buf.data_ptr() + (layer * 3 + which) * self.dim * buf.element_size()

    def _norm(self, start: int, **buffers) -> zero_block_norm_t:
        """Between layers start - 1 and start: the former's post-norm and gate, the latter's pre-norm."""
        last = start - 1
        args = zero_block_norm_t(rows=self.rows, dim=self.dim, dtype16=ZERO_BF16, kind=ZERO_NORM_RMS, eps=self.eps,
                                 residual_scale=1.0, **buffers)
        if start < self.layers:
            args.norms |= ZERO_NORM_PRE
            args.pre_w = self._vector(self.vectors16, start, 0)
        if last >= 0:
            args.norms |= ZERO_NORM_POST
            args.post_w = self._vector(self.vectors16, last, 1)
            args.gate, args.rows_per_gate = self._vector(self.vectors16, last, 2), self.rows
            args.residual_scale = self.scale
        return args

    # ------------------------------------------------------------------ forward, backward, step

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """x: rows x dim, bf16.  Keeps the activations that the backward pass reads."""
        s = self._stream()
        self.y[0].copy_(x)
        for l in range(self.layers + 1):
            if l == 0:
                zero_block_norm(self._norm(0, h=self.y[0].data_ptr(), z=self.z[0].data_ptr()), s)
            else:
                z = self.z[l].data_ptr() if l < self.layers else None
                zero_block_norm(self._norm(l, h=self.h[l - 1].data_ptr(), x=self.y[l - 1].data_ptr(),
                                           y=self.y[l].data_ptr(), z=z), s)
            if l == self.layers:
                break
            unit = self.unit16(l)
            for args in (self._linear(unit, l, False, x=self.z[l].data_ptr(), y=self.act[l].data_ptr(),
                                      pre=self.pre[l].data_ptr()),
                         self._linear(unit, l, True, x=self.act[l].data_ptr(), y=self.h[l].data_ptr())):
                n = zero_linear_workspace(args)
                zero_linear(args, self._room(n), n, s)
            self.group.release(l)
        return self.y[self.layers]

    def backward(self, rank: int, dy: torch.Tensor) -> None:
        """dy: the loss's gradient on the forward pass's result; rank's contributions are written."""
        s = self._stream()
        self.dy.copy_(dy)
        vectors = self.rank_vector_grads[rank]
        for l in range(self.layers, -1, -1):
            if l < self.layers:
                unit, grads = self.unit16(l), self.contribs[l][rank]
                base = grads.data_ptr()
                for args in (self._linear(unit, l, True, x=self.act[l].data_ptr(), dy=self.dh.data_ptr(),
                                          dx=self.da.data_ptr(), dw=base + 2 * self.at[2], dbias=base + 2 * self.at[3]),
                             self._linear(unit, l, False, x=self.z[l].data_ptr(), pre=self.pre[l].data_ptr(),
                                          dy=self.da.data_ptr(), dx=self.dz.data_ptr(), dw=base,
                                          dbias=base + 2 * self.at[1])):
                    n = zero_linear_workspace(args, True)
                    zero_linear_backward(args, self._room(n), n, s)
                self.group.release(l)
            args = self._norm(l, dy=self.dy.data_ptr(), dx=self.dy.data_ptr())
            if l < self.layers:
                args.y, args.dz = self.y[l].data_ptr(), self.dz.data_ptr()
                args.dpre_w = self._vector(vectors, l, 0)
            if l > 0:
                args.h, args.dh = self.h[l - 1].data_ptr(), self.dh.data_ptr()
                args.dpost_w, args.dgate = self._vector(vectors, l - 1, 1), self._vector(vectors, l - 1, 2)
            n = zero_block_norm_workspace(args)
            zero_block_norm_backward(args, self._room(n), n, s)

    def step(self, h) -> None:
        """One optimizer step from the ranks' gradients (no synchronisation): matrices and vectors are applied or
        left out together, and clipped by one norm."""
        contribs = [[c.data_ptr() for c in unit] for unit in self.contribs]
        torch.mean(self.rank_vector_grads.float(), 0, out=self.vector_grads)
        if h.max_grad_norm > 0:
            for u in range(self.layers):
                self.group.grad_norm(contribs[u], u)
        zero_adamw_check(self.opt, self.group.plan, self._stream())
        for u in range(self.layers):
            self.group.step(contribs[u], u, h)
        zero_adamw_step_with(self.opt, self.group.plan, h, self._stream())
        self.group.finish(wait=False)


def train(steps: int = 60, layers: int = 3, dim: int = 256, inner: int = 1024, n_d: int = 4, rows: int = 512,
          seed: int = 0) -> List[float]:
    """Fits a fixed random map of Gaussian tokens; the mean squared error after each step."""
    model = ShardedFeedForward(layers, dim, inner, n_d, rows, seed=seed)
    try:
        gen = torch.Generator(device="cuda").manual_seed(seed + 1)
        turn = torch.randn(dim, dim, generator=gen, device="cuda") * dim ** -0.5
        h = hyper(lr=2e-3, weight_decay=0.0)
        losses = []
        for _ in range(steps):
            total = torch.zeros((), device="cuda")
            for r in range(n_d):
                x = torch.randn(rows, dim, generator=gen, device="cuda").to(torch.bfloat16)
                want = x.float() + torch.tanh(x.float() @ turn)
                off = model.forward(x).float() - want
                total += off.square().mean() / n_d
                model.backward(r, (off * (2.0 / off.numel())).to(torch.bfloat16))
            model.step(h)
            losses.append(float(total))
        return losses
    finally:
        torch.cuda.synchronize()
        model.close()


if __name__ == "__main__":
    for i, loss in enumerate(train()):
        if i % 10 == 9 or i == 0:
            print(f"step {i + 1:3d}  mean squared error {loss:.4f}")
