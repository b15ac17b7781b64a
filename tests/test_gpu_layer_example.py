"""GPU test of the example that runs the operators together: one training step
of a mixture-of-experts block, against the same mathematics in 64 bits by
automatic differentiation, without quantization.

Tolerance: rounding to E4M3 is off by up to 2^-4 relative, 2.7 % in the root
mean square, a product of two such operands by 3.7 %.  The forward chains two
products (5.3 %) and the gradients of the up projection four (7.5 %, with the
forward's own errors in their operands below 10 %); 15 % in the 2-norm leaves
half again.
"""
import os
import sys

import pytest
import torch

import fp8_fine_grained_quantize_amd as fb

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_block_step as ex  # noqa: E402

pytestmark = pytest.mark.gpu

T, C, E, K, H = 300, 256, 8, 3, 128


def _rms(z, w):
    return z * torch.rsqrt(z.square().mean(1, keepdim=True) + 1e-6) * w


def _plain(b, x, experts):
    """x', n' in 64 bits, with the experts that the step chose."""
    p = {k: getattr(b, k).double().cpu().requires_grad_() for k in ("w_pre", "w_post", "gate", "w_next", "router", "up", "down")}
    x = x.double().cpu().requires_grad_()
    n = _rms(x, p["w_pre"])
    aff = torch.sigmoid(n @ p["router"]).gather(1, experts)
    w = aff / aff.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for e in range(E):
        t, k = torch.nonzero(experts == e, as_tuple=True)
        u = n[t] @ p["up"][e]
        o = (torch.nn.functional.silu(u[:, :H]) * u[:, H:]) @ p["down"][e]
        y = y.index_add(0, t, o * w[t, k][:, None])
    xo = x + ex.ALPHA * p["gate"] * _rms(y, p["w_post"])
    return xo, _rms(xo, p["w_next"]), x, p


def test_step_against_64_bits():
    b = ex.Block.random(C, E, K, H, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x, dx, dn = (torch.randn(T, C, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    xo, n, saved = ex.forward(b, x)
    got_dx, grads = ex.backward(b, saved, dx, dn)
    # the experts chosen, from the maps
    row_of, off = saved["row_of"].cpu().long(), saved["off"].cpu().long()
    experts = torch.bucketize(row_of, off[1:], right=True)
    pxo, pn, px, p = _plain(b, x, experts)
    (pxo * dx.double().cpu()).sum().add((pn * dn.double().cpu()).sum()).backward()
    for name, got, want in [("x", xo, pxo), ("n", n, pn), ("dx", got_dx, px.grad)] + \
            [(k, grads[k], p[k].grad) for k in p]:
        want = want.detach()
        err = float((got.double().cpu() - want).norm() / want.norm())
        print(f"[example] {name}: {err:.4f}", flush=True)
        assert err <= 0.15, name


def test_step_clips():
    b = ex.Block.random(C, E, K, H, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x, dx, dn = (torch.randn(T, C, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    _, _, _, grads, norm = ex.step(b, x, dx, dn, max_norm=0.5)
    assert float(norm) > 0.5
    assert abs(float(fb.grad_norm(list(grads.values()))) - 0.5) <= 1e-5


def test_command():
    ex.main(["--tokens", "64", "--hidden", "256", "--experts", "4", "--topk", "2", "--width", "128"])
