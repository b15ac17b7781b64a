"""GPU tests: the operators around the GEMMs run on the caller's stream, keep
nothing between calls and can be captured into a HIP graph.
"""
import pytest
import torch

import fp8_fine_grained_quantize_amd as fb

pytestmark = pytest.mark.gpu

T, K, E, C = 1500, 8, 256, 1032


def _bf16(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).cuda()


class _Step:
    """Static buffers of one step through every operator, outputs given."""

    def __init__(self, seed):
        self.x, self.f, self.gate = _bf16((T, C), seed), _bf16((T, C), seed + 1), _bf16((C,), seed + 2)
        self.w = (1 + 0.1 * _bf16((C,), seed + 3)).contiguous()
        self.ids = torch.empty(T, K, dtype=torch.int64, device="cuda")
        self.p = torch.empty(T, K, device="cuda")
        self.fill(seed)
        self.table = fb.grad_table([self.f, self.p], [torch.empty(T, C, device="cuda"), torch.empty(T, K, device="cuda")])

    def fill(self, seed):
        g = torch.Generator().manual_seed(seed + 4)
        self.x.copy_(_bf16((T, C), seed))
        self.ids.copy_(torch.randint(-1, E + 1, (T, K), generator=g))
        self.p.copy_(torch.rand(T, K, generator=g))

    def run(self):
        r = fb.residual_norm(self.x, w_pre=self.w, f=self.f, w_post=self.w, gate=self.gate, alpha=0.5, quantize=True)
        off, row_of, slot_of = fb.moe_sort(self.ids, E)
        qr, sr = fb.moe_dispatch_fp8(r.q, r.s, row_of, slot_of)
        rows = fb.moe_dispatch(r.n, row_of)
        y = fb.moe_combine(rows, row_of, self.p)
        dr, dw = fb.moe_combine_backward(r.n, rows, row_of, self.p)
        g = fb.residual_norm_backward(r.x, dx_out=y, dn=r.n, rstd_pre=r.rstd_pre, w_pre=self.w, f=self.f,
                                      rstd_post=r.rstd_post, w_post=self.w, gate=self.gate, alpha=0.5)
        norm = fb.clip_grad_norm(self.table, 3.0)
        return [*r, off, row_of, slot_of, qr, sr, rows, y, dr, dw, *g, norm, *self.table.outs]


def _same(a, b):
    return len(a) == len(b) and all(torch.equal(p, q) for p, q in zip(a, b))


def test_two_streams_equal_sequential():
    one, two = _Step(1), _Step(50)
    ref = [[t.clone() for t in s.run()] for s in (one, two)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(s1):
            a = one.run()
        with torch.cuda.stream(s2):
            b = two.run()
        torch.cuda.synchronize()
        assert _same(a, ref[0]) and _same(b, ref[1])


def test_graph_replays_equal_eager():
    step = _Step(7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    print("[layer] capture", flush=True)
    with torch.cuda.graph(graph):
        out = step.run()
    torch.cuda.synchronize()
    other = _Step(90)
    for rep in range(4):
        if rep in (1, 3):
            step.fill(100 + rep)
            torch.cuda.synchronize()
        print(f"[layer] replay {rep}", flush=True)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert _same(got, step.run()), rep
        other.run()
        torch.cuda.synchronize()
