"""One training step of a mixture-of-experts block in FP8: forward, backward,
gradient clipping and the optimizer's update, every step of it a call of this
package (the router's product and top-k are torch).

    python examples/moe_block_step.py [--tokens 8192 --hidden 7168 --experts 256 --topk 8 --width 2048]

Forward, for the residual stream x:
    n         = norm before the block, with its 1x128 codes       residual_norm
    experts   = top-k of sigmoid(n Wr), weights normalized        torch
    maps      = pairs sorted by expert                            moe_sort
    rows      = codes and scales in expert order                  moe_dispatch_fp8
    u, h      = gate and up projection, h = silu(gate) * up       grouped_gated_gemm_fp8_blockscaled
    o         = down projection of h's codes                      grouped_gemm_fp8_blockscaled
    y         = rows back to tokens, weighted                     moe_combine
    x', n'    = norm of y, gate, residual sum, next block's norm  residual_norm
Backward, from the gradients of x' and n', the same in reverse; quantization
passes gradients through.  Between the two, only u is kept of an expert's rows:
the gradient of the down projection's input, the activation's gradient and h
from u are one call (grouped_gated_gemm_backward_fp8_blockscaled), which leaves
the gradient in u's memory: a backward pass uses up what its forward kept.

Update: AdamW with E4M3 moments on the FP32 norms and router and on the BF16
expert weights (rounded at random), gradients clipped by their global norm as
they are read; then the expert weights' codes anew.
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import fp8_fine_grained_quantize_amd as fb  # noqa: E402

ALPHA = 0.5  # the block's residual scale


@dataclass
class Block:
    """Parameters of one block; expert weights also as FP8 codes and 128x128 scales."""
    w_pre: torch.Tensor    # [C] norm before the block
    w_post: torch.Tensor   # [C] norm after it
    gate: torch.Tensor     # [C] gate on the normed output
    w_next: torch.Tensor   # [C] norm before the next block
    router: torch.Tensor   # [C][E]
    up: torch.Tensor       # [E][C][2H]
    down: torch.Tensor     # [E][H][C]
    topk: int

    def __post_init__(self):
        self.quantize()

    def quantize(self):
        self.q_up, self.s_up = self._quantize(self.up)
        self.q_down, self.s_down = self._quantize(self.down)

    @staticmethod
    def _quantize(w):
        E, R, C = w.shape  # R a multiple of 128: the stacked blocks are each expert's own
        q, s = fb.quantize_block128(w.view(E * R, C))
        return q.view(E, R, C), s.view(E, R // 128, -1)

    @staticmethod
    def random(C, E, topk, H, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        return Block(w_pre=1 + 0.1 * n(C), w_post=1 + 0.1 * n(C), gate=0.8 + 0.1 * n(C), w_next=1 + 0.1 * n(C),
                     router=n(C, E) * C ** -0.5,
                     up=torch.stack([(n(C, 2 * H) * C ** -0.5).to(torch.bfloat16) for _ in range(E)]),
                     down=torch.stack([(n(H, C) * H ** -0.5).to(torch.bfloat16) for _ in range(E)]), topk=topk)


NAMES = ("w_pre", "w_post", "gate", "w_next", "router", "up", "down")


class Optimizer:
    """AdamW over a block's parameters; no weight decay on norms and gate."""

    def __init__(self, b: Block, lr=1e-3, max_norm=1.0):
        self.block, self.lr, self.max_norm, self.steps = b, lr, max_norm, 0
        self.state = fb.AdamWState([getattr(b, k) for k in NAMES], dtype=torch.float8_e4m3fn,
                                   decay=[0.1 if k in ("router", "up", "down") else 0.0 for k in NAMES])

    def update(self, grads) -> torch.Tensor:
        """One step from gradients by name; returns their norm before clipping."""
        self.steps += 1
        grads = [grads[k] for k in NAMES]
        norm = fb.grad_norm(grads)
        fb.adamw_step(fb.adamw_table(self.state, grads), self.lr, self.steps, norm=norm, max_norm=self.max_norm,
                      seed=self.steps)
        self.block.quantize()
        return norm


def forward(b: Block, x: torch.Tensor):
    """(x', n', what the backward needs)."""
    E = b.up.shape[0]
    r0 = fb.residual_norm(x, w_pre=b.w_pre, quantize=True)
    n_router = r0.n.float().requires_grad_()
    router = b.router.detach().requires_grad_()
    with torch.enable_grad():
        top = torch.topk(torch.sigmoid(n_router @ router), b.topk, dim=1)
        weights = top.values / top.values.sum(1, keepdim=True)
    off, row_of, slot_of = fb.moe_sort(top.indices, E)
    qx, sx = fb.moe_dispatch_fp8(r0.q, r0.s, row_of, slot_of)
    r = fb.grouped_gated_gemm_fp8_blockscaled(off, qx, sx, b.q_up, b.s_up, quantize=True, want_h=False)
    o = fb.grouped_gemm_fp8_blockscaled(off, r.q, r.s, b.q_down, b.s_down)
    w = weights.detach()
    y = fb.moe_combine(o, row_of, w)
    r1 = fb.residual_norm(x, w_pre=b.w_next, f=y, w_post=b.w_post, gate=b.gate, alpha=ALPHA)
    return r1.x, r1.n, dict(x=x, r0=r0, n_router=n_router, router=router, weights=weights, w=w, off=off, row_of=row_of,
                            u=r.u, o=o, y=y, r1=r1)


def backward(b: Block, s: dict, dx_out: torch.Tensor, dn: torch.Tensor):
    """(dx, gradients by name) from the gradients of x' and n'."""
    off, row_of, r0, r1 = s["off"], s["row_of"], s["r0"], s["r1"]
    P = row_of.numel()
    g1 = fb.residual_norm_backward(r1.x, dx_out=dx_out, dn=dn, rstd_pre=r1.rstd_pre, w_pre=b.w_next, f=s["y"],
                                   rstd_post=r1.rstd_post, w_post=b.w_post, gate=b.gate, alpha=ALPHA)
    do, dweights = fb.moe_combine_backward(g1.df, s["o"], row_of, s["w"], drows_dtype=torch.bfloat16)
    # down projection and activation: gradient of u (in its place) with its codes, and h from u
    g = fb.grouped_gated_gemm_backward_fp8_blockscaled(off, *fb.quantize_1x128(do), b.q_down, b.s_down, s["u"],
                                                       quantize=True, du=s["u"])
    d_down = fb.grouped_wgrad_fp8_blockscaled(off, P, *fb.quantize_128x1_grouped(g.h, off),
                                              *fb.quantize_128x1_grouped(do, off))
    # up projection
    dxr = fb.grouped_gemm_fp8_blockscaled(off, g.q, g.s, b.q_up, b.s_up, opB=fb.OP_T, out_dtype=torch.bfloat16)
    rows = fb.moe_dispatch(r0.n, row_of)
    d_up = fb.grouped_wgrad_fp8_blockscaled(off, P, *fb.quantize_128x1_grouped(rows, off),
                                            *fb.quantize_128x1_grouped(g.du, off))
    # the router, and the norm before the block
    s["weights"].backward(dweights)
    dn0 = fb.moe_combine(dxr, row_of, out_dtype=torch.float32).add_(s["n_router"].grad).to(torch.bfloat16)
    g0 = fb.residual_norm_backward(s["x"], dx_out=g1.dx, dn=dn0, rstd_pre=r0.rstd_pre, w_pre=b.w_pre)
    return g0.dx, dict(w_pre=g0.dw_pre, w_post=g1.dw_post, gate=g1.dgate, w_next=g1.dw_pre, router=s["router"].grad,
                       up=d_up, down=d_down)


def step(b: Block, x, dx_out, dn, max_norm=1.0):
    """Forward, backward and clipping: (x', n', dx, clipped gradients, their norm before)."""
    xo, n, saved = forward(b, x)
    dx, grads = backward(b, saved, dx_out, dn)
    norm = fb.clip_grad_norm(list(grads.values()), max_norm)
    return xo, n, dx, grads, norm


def train_step(b: Block, opt: Optimizer, x, dx_out, dn):
    """Forward, backward and update: (x', n', dx, the gradients' norm before clipping)."""
    xo, n, saved = forward(b, x)
    dx, grads = backward(b, saved, dx_out, dn)
    return xo, n, dx, opt.update(grads)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--topk", type=int, default=8)
    ap.add_argument("--width", type=int, default=1024)
    a = ap.parse_args(argv)
    b = Block.random(a.hidden, a.experts, a.topk, a.width)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dx, dn = (torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16) * k
                 for k in (1.0, 1e-3, 1e-3))
    opt = Optimizer(b)
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(4):
        t0.record()
        _, _, _, norm = train_step(b, opt, x, dx, dn)
        t1.record()
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens, hidden {a.hidden}, {a.experts} experts of width {a.width}, top {a.topk}: "
          f"{t0.elapsed_time(t1):.2f} ms a step, gradient norm {float(norm):.4g} over "
          f"{sum(getattr(b, k).numel() for k in NAMES)} values")


if __name__ == "__main__":
    main()
