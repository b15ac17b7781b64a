"""GPU tests of the example's training step with its update: the operators of a whole step, one after the other.

The gradients themselves are held against 64 bits in test_gpu_layer_example.py.
"""
import os
import sys

import numpy as np
import pytest
import torch

import fp8_fine_grained_quantize_amd as fb
from tests import train_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_block_step as ex  # noqa: E402

pytestmark = pytest.mark.gpu

T, C, E, K, H = 300, 256, 8, 3, 128


def _inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(T, C, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]


def _np(t):
    return t.detach().cpu().double().numpy().reshape(-1)


def test_update_is_adamw_of_the_gradients():
    """Every parameter after a step, from the gradients that the step saw, within the bounds of one AdamW step; the
    codes are those of the new weights."""
    b = ex.Block.random(C, E, K, H, seed=3)
    opt = ex.Optimizer(b, lr=1e-2, max_norm=0.5)
    for steps in (1, 2):
        x, dx, dn = _inputs(10 + steps)
        _, _, saved = ex.forward(b, x)
        _, grads = ex.backward(b, saved, dx, dn)
        old = [_np(getattr(b, k)) for k in ex.NAMES]
        s = opt.state
        m, v = [], []
        for i, p in enumerate(s.params):
            n = p.numel()
            m.append(ref.decode(s.ms[i].cpu().numpy()) * ref.spread(_np(s.m_scales[i]), n))
            v.append((ref.decode(s.vs[i].cpu().numpy()) * ref.spread(_np(s.v_scales[i]), n)) ** 2)
        norm = float(opt.update(grads))
        clip = min(1.0, 0.5 / (norm + 1e-6))
        for i, k in enumerate(ex.NAMES):
            p = getattr(b, k)
            want, e = ref.adamw(old[i], _np(grads[k]), m[i], v[i], 1e-2, steps, 0.9, 0.95, 1e-8, s.decay[i], clip)["p"]
            bound = ref.bf16_bound(want, e, True) if p.dtype == torch.bfloat16 else e
            assert np.all(np.abs(_np(p) - want) <= bound), (steps, k)
        q, sc = fb.quantize_block128(b.up.view(E * C, 2 * H))
        assert torch.equal(b.q_up.view(E * C, 2 * H), q) and torch.equal(b.s_up.view(-1), sc.view(-1))
    assert opt.steps == 2


def test_steps_repeat():
    """Two blocks of the same seed: the same bits after three steps."""
    ends = []
    for _ in range(2):
        b = ex.Block.random(C, E, K, H, seed=5)
        opt = ex.Optimizer(b)
        for i in range(3):
            out = ex.train_step(b, opt, *_inputs(20 + i))
        ends.append([*out, *(getattr(b, k) for k in ex.NAMES), *opt.state.ms, *opt.state.vs])
    assert all(torch.equal(p, q) for p, q in zip(*ends))


def test_operators_of_one_layer_on_two_streams():
    """The block's forward and backward on two streams at once equals one after the other."""
    blocks = [ex.Block.random(C, E, K, H, seed=s) for s in (1, 2)]
    ins = [_inputs(s) for s in (30, 40)]

    def run(b, x, dx, dn):
        xo, n, saved = ex.forward(b, x)
        g, grads = ex.backward(b, saved, dx, dn)
        return [xo, n, g, *(grads[k] for k in ex.NAMES)]

    want = [[t.clone() for t in run(b, *i)] for b, i in zip(blocks, ins)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for s, b, i in zip(streams, blocks, ins):
        with torch.cuda.stream(s):
            got.append(run(b, *i))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(w, g))
