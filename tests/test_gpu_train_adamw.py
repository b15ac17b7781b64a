"""GPU tests of the AdamW step over many tensors, against 64-bit forms with the
bounds of train_ref.py.
"""
import math

import numpy as np
import pytest
import torch

import fp8_fine_grained_quantize_amd as fb
from tests import train_ref as ref
from tests.layer_ref import U, UB

pytestmark = pytest.mark.gpu

LR, B1, B2, EPS = 3e-3, 0.9, 0.95, 1e-8
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _np(t):
    return t.detach().cpu().double().numpy().reshape(-1)


def _rand(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def _moments(sizes, kind, seed):
    """Moments of a training run under way, of both signs, zeros among them."""
    kw = dict(ms=[], vs=[])
    if kind == E4:
        kw.update(m_scales=[], v_scales=[])
    for i, n in enumerate(sizes):
        m, v = _rand(n, F32, seed + 3 * i, 1e-2), _rand(n, F32, seed + 3 * i + 1, 1e-2).square()
        m[::17], v[::19] = 0, 0
        if kind != E4:
            kw["ms"].append(m.to(kind))
            kw["vs"].append(v.to(kind))
            continue
        for x, q, s in ((m, "ms", "m_scales"), (v.sqrt(), "vs", "v_scales")):
            G = -(-n // 128)
            t = torch.nn.functional.pad(x, (0, G * 128 - n)).view(G, 128)
            sc = torch.clamp(t.abs().amax(1), min=1e-20) / 448 if G else t.new_zeros(0)
            kw[q].append((t / sc[:, None]).clamp(-448, 448).to(E4).view(torch.uint8).view(-1)[:n].clone())
            kw[s].append(sc)
    return kw


def _stored(s, i):
    """(m, v) of tensor i as the state holds them."""
    m, v = s.ms[i].cpu().numpy() if s.state == 2 else _np(s.ms[i]), s.vs[i].cpu().numpy() if s.state == 2 else _np(s.vs[i])
    if s.state != 2:
        return m, v
    n = m.size
    return ref.decode(m) * ref.spread(_np(s.m_scales[i]), n), (ref.decode(v) * ref.spread(_np(s.v_scales[i]), n)) ** 2


def _flat(t, like):
    """Elements in the order that `like` has in memory."""
    order = sorted(range(like.dim()), key=lambda d: -like.stride(d))
    return _np(t.permute(order))


def _check(s, before, grads, clip, random, step, lr=LR, b1=B1, b2=B2, eps=EPS):
    for i, p in enumerate(s.params):
        if p.numel() == 0:
            continue
        p0, (m0, v0) = before[i]
        want = ref.adamw(p0, _flat(grads[i], p), m0, v0, lr, step, b1, b2, eps, s.decay[i], clip)
        p1, ep = want["p"]
        got = _flat(p, p)
        assert np.all(np.abs(got - p1) <= (ep if p.dtype == F32 else ref.bf16_bound(p1, ep, random))), (i, "p")
        if s.copies[i] is not None:
            assert np.all(np.abs(_flat(s.copies[i], p) - p1) <= ref.bf16_bound(p1, ep, False)), (i, "copy")
        for name, q, sc in (("m", s.ms, s.m_scales), ("v", s.vs, s.v_scales)):
            x, e = want[name]
            if s.state == 0:
                assert np.all(np.abs(_np(q[i]) - x) <= e), (i, name)
            elif s.state == 1:
                assert np.all(np.abs(_np(q[i]) - x) <= ref.bf16_bound(x, e, random)), (i, name)
            else:
                x, e = want["r"] if name == "v" else (x, e)
                scale, es, b = ref.code_bounds(x, e, random, name == "v")
                assert np.all(np.abs(_np(sc[i]) - scale) <= es), (i, name, "scale")
                val = ref.decode(q[i].cpu().numpy()) * ref.spread(_np(sc[i]), x.size)
                assert np.all(np.abs(val - x) <= b), (i, name)
                if name == "v":
                    assert np.all((val > 0) == (x > 0)), i


SIZES = [1, 3, 4, 127, 128, 129, 1023, 1024, 1025, 2047, 2048, 2049, 5000, 0, 20001]


@pytest.mark.parametrize("kind", [F32, BF, E4])
@pytest.mark.parametrize("pt,gt", [(F32, F32), (F32, BF), (BF, F32), (BF, BF)])
@pytest.mark.parametrize("random", [False, True])
def test_step(kind, pt, gt, random):
    print(f"[train] adamw {kind} {pt} {gt} {random}", flush=True)
    params = [_rand(n, pt, i) for i, n in enumerate(SIZES)]
    grads = [_rand(n, gt, 50 + i, 1e-2) for i, n in enumerate(SIZES)]
    if len(grads[12]):
        grads[12][100:300] = 0
    copies = [torch.empty(n, dtype=BF, device="cuda") for n in SIZES]
    s = fb.AdamWState(params, **_moments(SIZES, kind, 100), copies=copies, decay=[0.1 * (i % 3) for i in range(len(SIZES))])
    table = fb.adamw_table(s, grads)
    kept = [g.clone() for g in grads]
    for step in (1, 2, 1000):
        before = [(_np(p), _stored(s, i)) for i, p in enumerate(params)]
        norm = fb.grad_norm(grads) if step > 1 else None
        kw = {} if norm is None else dict(norm=norm, max_norm=0.5 * float(norm))
        fb.adamw_step(table, LR, step, beta1=B1, beta2=B2, eps=EPS, seed=77 + step if random else None, **kw)
        clip = 1.0 if norm is None else min(1.0, 0.5 * float(norm) / (float(norm) + 1e-6))
        _check(s, before, grads, clip, random, step)
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))


def test_many_small_and_one_large():
    """More entries than a search step holds, and chunks shared out over every workgroup."""
    sizes = [(i * 37) % 300 + 1 for i in range(700)] + [3000017]
    params, grads = [_rand(n, F32, i) for i, n in enumerate(sizes)], [_rand(n, BF, 9000 + i) for i, n in enumerate(sizes)]
    s = fb.AdamWState(params, decay=0.1)
    before = [(_np(p), _stored(s, i)) for i, p in enumerate(params)]
    fb.adamw_step(fb.adamw_table(s, grads), LR, 1, eps=EPS)
    _check(s, before, grads, 1.0, False, 1)


@pytest.mark.parametrize("kind", [F32, BF, E4])
@pytest.mark.parametrize("cols", [20, 21, 128, 1])
def test_rows_apart(kind, cols):
    """Parameters, gradients and copies whose rows lie apart; what lies between stays."""
    R = 157
    base_p, base_c = _rand((R, cols + 7), F32, 1), _rand((R, cols + 3), BF, 2)
    p, c, g = base_p[:, 2:2 + cols], base_c[:, :cols], _rand((R, cols + 4), F32, 3)[:, 1:1 + cols]
    old_p, old_c = base_p.clone(), base_c.clone()
    s = fb.AdamWState([p], **_moments([R * cols], kind, 5), copies=[c], decay=0.1)
    before = [(_np(p), _stored(s, 0))]
    fb.adamw_step(fb.adamw_table(s, [g]), LR, 3, eps=EPS)
    _check(s, before, [g], 1.0, False, 3)
    assert torch.equal(base_p[:, :2], old_p[:, :2]) and torch.equal(base_p[:, 2 + cols:], old_p[:, 2 + cols:])
    assert torch.equal(base_c[:, cols:], old_c[:, cols:])


def test_transposed_and_unaligned():
    p, g = _rand((60, 33), F32, 1).t(), _rand((60, 33), BF, 2).t()
    flat, gf = _rand(5003, BF, 3), _rand(5004, F32, 4)
    s = fb.AdamWState([p, flat[1:]], decay=0.1)
    before = [(_flat(p, p), _stored(s, 0)), (_np(flat[1:]), _stored(s, 1))]
    fb.adamw_step(fb.adamw_table(s, [g, gf[2:]]), LR, 3, eps=EPS)
    _check(s, before, [g, gf[2:]], 1.0, False, 3)


def test_random_bf16_as_defined():
    """Moments and parameters whose FP32 values are known: beta 0 gives m = g and
    v = g^2; with one step, eps 0 and a root that is exact, p moves by lr."""
    n = 5001
    g = (torch.arange(1, n + 1).float() * 3.0)  # at most 14 bits: g^2 and its root are exact
    g[::2] *= -1
    p = torch.zeros(n, dtype=BF, device="cuda")
    first = fb.AdamWState([torch.zeros(4, device="cuda"), p], dtype=BF)
    fb.adamw_step(fb.adamw_table(first, [torch.zeros(4, device="cuda"), g.cuda()]), 0.3, 1, beta1=0.0, beta2=0.0, eps=0.0,
                  seed=12345)
    key, at = ref.key_of(12345, 1), np.arange(n)
    r, rp = ref.random_bits(key, at), ref.random_bits(key ^ 0x5BD1E995, at)
    gn = g.numpy()
    assert np.array_equal(_np(first.ms[1]), ref.drop(gn, 16, r & 0xFFFF).astype(np.float64))
    assert np.array_equal(_np(first.vs[1]), ref.drop(gn * gn, 16, r >> 16).astype(np.float64))
    want = -np.sign(gn) * np.float32(0.3)
    assert np.array_equal(_np(p), ref.drop(want, 16, rp & 0xFFFF).astype(np.float64))
    assert len(np.unique(_np(p))) == 4


def test_random_codes_as_defined():
    """Groups whose largest value is 448 times a power of two: the quotients are exact."""
    n = 128 * 40 + 57
    rng = np.random.RandomState(1)
    g = (rng.randn(n) * np.exp2(rng.randint(-16, 4, n))).astype(np.float32)
    g = np.clip(g, -400, 400)
    g[::128] = 448.0
    g[5::128] = 0.0
    s = fb.AdamWState([torch.zeros(n, device="cuda")], dtype=E4)
    fb.adamw_step(fb.adamw_table(s, [torch.from_numpy(g).cuda()]), 0.0, 1, beta1=0.0, beta2=0.0, seed=99)
    r = ref.random_bits(ref.key_of(99), np.arange(n))

    def codes(x, r16, floor):
        a = np.abs(x).astype(np.float32)
        up = np.where(a < 2.0 ** -6, np.float32(2.0 ** -6), np.float32(0))
        a = ref.drop(a + up, 20, r16 << 4) - up
        if floor:
            a = np.where((x > 0) & (a == 0), np.float32(2.0 ** -9), a)
        return np.copysign(a, x).astype(np.float64)

    assert np.all(_np(s.m_scales[0]) == 1.0)
    assert np.array_equal(ref.decode(s.ms[0].cpu().numpy()), codes(g, r & 0xFFFF, False))
    root = np.sqrt((g * g).astype(np.float32))  # correctly rounded in both
    assert np.array_equal(ref.decode(s.vs[0].cpu().numpy()), codes(root, r >> 16, True))


@pytest.mark.parametrize("kind", [BF, E4])
def test_random_keeps_small_changes(kind):
    """The mean over seeds of what is stored lies at the value itself.  A value between two codes
    q apart is stored with a variance of at most q^2 / 4, so that the mean of N is off by at most
    6 q / (2 sqrt(N)) but for one in 10^9; the 16 bits give the probability to 2^-16."""
    n, N = 1280, 256
    g = _rand(n, F32, 3).abs() + 0.5
    total = torch.zeros(n, dtype=torch.float64)
    for seed in range(N):
        s = fb.AdamWState([torch.zeros(n, device="cuda")], dtype=kind)
        fb.adamw_step(fb.adamw_table(s, [g]), 0.0, 1, beta1=0.0, beta2=0.5, seed=1000003 * seed)
        total += torch.from_numpy(_stored(s, 0)[0])
    x = _np(g)
    q = (2 * UB if kind == BF else 2.0 ** -3) * x * (1 + 2.0 ** -10)
    assert np.all(np.abs(total.numpy() / N - x) <= q * (3 / math.sqrt(N) + 2.0 ** -15) + 4 * U * x)


def test_edges():
    """Zeros, infinities and NaN stay in their element (FP32) or its 128 (codes);
    a norm of infinity takes nothing, a NaN norm spoils all."""
    n = 384
    p, g = _rand(n, F32, 1), _rand(n, F32, 2)
    g[:128] = 0
    g[130], g[131] = math.inf, math.nan
    for kind in (F32, E4):
        s = fb.AdamWState([p.clone()], dtype=kind)
        t = fb.adamw_table(s, [g])
        fb.adamw_step(t, LR, 1)
        bad = ~torch.isfinite(s.params[0])
        assert bad.nonzero().view(-1).tolist() == [130, 131]
        assert torch.equal(s.params[0][:128], p[:128])      # 0 / (0 + eps)
        if kind == E4:
            assert float(s.m_scales[0][0]) == 1.0 and not s.ms[0][:128].any() and not s.vs[0][:128].any()
            assert math.isnan(float(s.m_scales[0][1])) and math.isfinite(float(s.m_scales[0][2]))
            fb.adamw_step(t, LR, 2)
            assert torch.isfinite(s.params[0][256:]).all()
    z = fb.AdamWState([p.clone()])
    fin = torch.where(torch.isfinite(g), g, torch.zeros_like(g))
    fb.adamw_step(fb.adamw_table(z, [fin]), LR, 1, norm=torch.tensor(math.inf, device="cuda"), max_norm=1.0)
    assert torch.equal(z.params[0], p) and not z.ms[0].any()
    fb.adamw_step(fb.adamw_table(z, [fin]), LR, 1, norm=torch.tensor(math.nan, device="cuda"), max_norm=1.0)
    assert torch.isnan(z.params[0]).all()
    e = fb.AdamWState([])
    fb.adamw_step(fb.adamw_table(e, []), LR, 1)


def test_tiny_and_huge_moments():
    """Codes over the whole range of FP32's exponents."""
    n = 128 * 6
    g = _rand(n, F32, 4)
    for k, e in enumerate((1e-30, 1e-18, 1e-9, 1.0, 1e9, 1e17)):
        g[128 * k:128 * (k + 1)] *= e
    s = fb.AdamWState([torch.zeros(n, device="cuda")], dtype=E4)
    before = [(np.zeros(n), _stored(s, 0))]
    fb.adamw_step(fb.adamw_table(s, [g]), LR, 1, beta1=B1, beta2=B2, eps=1e-20)
    _check(s, before, [g], 1.0, False, 1, eps=1e-20)


def test_roots_are_rounded_correctly():
    """The root of every moment from the smallest subnormal on: p = -1 / sqrt(v) where m = 1, in FP32 bit for bit."""
    g = torch.Generator().manual_seed(3)
    n = 1 << 20
    bits = torch.randint(1, 0x7F000000, (n,), generator=g, dtype=torch.int64)  # halves of finite values
    bits[:64] = torch.arange(1, 65)
    bits[64:4160] = 0x0D800000 - 2048 + torch.arange(4096)  # around 2^-100
    x = bits.to(torch.int32).view(F32)
    x[4160:4160 + 4096] = torch.arange(1, 4097).float() ** 2 * 2.0 ** -60  # exact roots, and their neighbours
    x[9000:9000 + 4096] = torch.nextafter(x[4160:4160 + 4096], torch.tensor(3e38))
    p = torch.zeros(n, device="cuda")
    s = fb.AdamWState([p], [torch.full((n,), 2.0, device="cuda")], [(2 * x.double()).float().cuda()])
    fb.adamw_step(fb.adamw_table(s, [torch.zeros(n, device="cuda")]), 1.0, 10000, beta1=0.5, beta2=0.5, eps=0.0)
    assert torch.equal(s.vs[0].cpu(), x) and (s.ms[0] == 1).all()
    want = -(np.float32(1) / np.sqrt(x.numpy()))
    assert want.dtype == np.float32 and np.array_equal(p.cpu().numpy(), want)


def test_refusals_on_the_gpu():
    p, g = torch.zeros(8, device="cuda"), torch.zeros(8, device="cuda")
    t = fb.adamw_table(fb.AdamWState([p]), [g])
    one = torch.ones((), device="cuda")
    for kw in (dict(lr=math.nan), dict(step=0), dict(beta1=1.0), dict(beta2=-0.5), dict(eps=-1.0), dict(norm=one, max_norm=-1.0)):
        with pytest.raises(fb.Fp8BlkError):
            fb.adamw_step(t, **{"lr": 1e-3, "step": 1, **kw})
    for kw in (dict(norm=one), dict(max_norm=1.0), dict(norm=torch.ones(2, device="cuda"), max_norm=1.0),
               dict(lr=torch.ones(2, device="cuda")), dict(norm=torch.ones(()), max_norm=1.0),
               dict(step=torch.ones(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            fb.adamw_step(t, **{"lr": 1e-3, "step": 1, **kw})
    for kw in (dict(lr=one.double()), dict(step=one), dict(seed=one), dict(norm=one.double(), max_norm=1.0), dict(lr="x"),
               dict(step=1.5)):
        with pytest.raises(TypeError):
            fb.adamw_step(t, **{"lr": 1e-3, "step": 1, **kw})
    with pytest.raises(ValueError, match="share memory"):
        fb.adamw_table(fb.AdamWState([p, p]), [g, g])
    assert not p.any()


def test_streams_and_graph():
    """A step captured with its values in device memory equals eager steps at every replay."""
    sizes = [5000, 77, 300000]

    def fresh():
        kw = _moments(sizes, E4, 60)
        s = fb.AdamWState([_rand(n, BF, i) for i, n in enumerate(sizes)], **kw, decay=0.1)
        grads = [_rand(n, F32, 40 + i, 1e-2) for i, n in enumerate(sizes)]
        return s, grads, fb.adamw_table(s, grads)

    def all_of(s):
        return [t for ts in (s.params, s.ms, s.vs, s.m_scales, s.v_scales) for t in ts]

    def eager(tab, k, v):
        n = fb.grad_norm(tab.grads)
        fb.adamw_step(tab, v, k, norm=n, max_norm=0.1, seed=17 * k)

    a, ga, ta = fresh()
    b, gb, tb = fresh()
    lr = torch.zeros((), device="cuda")
    step, seed = (torch.zeros((), dtype=torch.int64, device="cuda") for _ in range(2))
    norms = fb.grad_table(ga)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step.add_(1)
        seed.add_(17)
        fb.adamw_step(ta, lr, step, norm=fb.grad_norm(norms), max_norm=0.1, seed=seed)
    for k in range(1, 6):
        value = float(np.float32(1e-2 / k))
        lr.fill_(value)
        for x, y in zip(ga, gb):
            x.mul_(0.9)
            y.mul_(0.9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        if k % 2:
            eager(tb, k, value)
        else:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                eager(tb, k, value)
        torch.cuda.synchronize()
        # the powers of beta come from two libraries (FP64, a few units in the last place): one FP32 step
        # size may be the neighbour of the other, and where it is, values may be stored apart
        same = [torch.equal(x, y) for x, y in zip(all_of(a), all_of(b))]
        assert all(same), (k, same)


@pytest.mark.parametrize("kind", [F32, BF, E4])
@pytest.mark.parametrize("pt,gt", [(F32, BF), (BF, F32)])
@pytest.mark.parametrize("large", [17_000_003, 36_000_131])
def test_many_chunks_of_a_workgroup(kind, pt, gt, large):
    """A table whose workgroups take several chunks, cached and streamed: the bits that its parts get in short tables."""
    print(f"[train] adamw many chunks {kind} {pt} {gt} {large}", flush=True)
    sizes = [large] + [1024 * k + d for k in range(7) for d in (1, 1023, 500)]
    gen = torch.Generator(device="cuda").manual_seed(5)
    P = [torch.randn(n, generator=gen, device="cuda").to(pt) for n in sizes]
    G = [(torch.randn(n, generator=gen, device="cuda") * 1e-2).to(gt) for n in sizes]
    C = [torch.zeros(n, dtype=BF, device="cuda") for n in sizes]

    def step(p, c, g):
        s = fb.AdamWState(p, dtype=kind, decay=0.1, copies=c)
        t = fb.adamw_table(s, g)
        for k in (1, 2):
            fb.adamw_step(t, LR, k, beta1=B1, beta2=B2, eps=EPS)
        return [t for part in zip(*(x for x in (p, s.ms, s.vs, c, s.m_scales, s.v_scales) if x[0] is not None)) for t in part]

    first, part = [p.clone() for p in P], 1024 * 4000
    cuts = [list(torch.split(x[0], part)) for x in (first, C, G)]
    got = step(P, C, G)
    per = len(got) // len(sizes)
    want = step(first[1:], [torch.zeros_like(c) for c in C[1:]], G[1:])
    assert all(torch.equal(a, b) for a, b in zip(got[per:], want))
    whole = got[:per]  # the large one's, against its pieces
    for i, (p, c, g) in enumerate(zip(*cuts)):
        for whole_t, t in zip(whole, step([p], [torch.zeros_like(c)], [g])):
            lo = i * (part if whole_t.numel() == large else part // 128)
            assert torch.equal(whole_t[lo:lo + t.numel()], t), (i, t.dtype)


@pytest.mark.parametrize("kind", [BF, E4])
def test_past_32_bits(kind):
    """The end of a tensor of more than 2^32 bytes equals the same values in a short one."""
    n, tail = 2 ** 31 + 128 * 9, 128 * 1000
    p, g = torch.zeros(n, dtype=BF, device="cuda"), torch.zeros(n, dtype=BF, device="cuda")
    p[-tail:], g[-tail:] = _rand(tail, BF, 1), _rand(tail, BF, 2)
    long = fb.AdamWState([p], dtype=kind, decay=0.1)
    short = fb.AdamWState([p[-tail:].clone()], dtype=kind, decay=0.1)
    for s, gr in ((long, g), (short, g[-tail:].clone())):
        t = fb.adamw_table(s, [gr])
        for k in (1, 2):
            fb.adamw_step(t, LR, k)
    assert torch.equal(long.params[0][-tail:], short.params[0]) and not long.params[0][:-tail].any()
    assert torch.equal(long.ms[0][-tail:], short.ms[0]) and torch.equal(long.vs[0][-tail:], short.vs[0])
