"""GPU tests of residual_norm and its gradient against the plain 64-bit forms
of layer_ref.py, with the bounds derived there.

A sum over the C channels of a row has C terms, so a statistic's relative
error is at most C U / 2 + 4 U (half of the sum's, then the division, the
square root, the scaling and the quotient); the bounds below double it.
"""
import itertools

import numpy as np
import pytest
import torch

import fp8_fine_grained_quantize_amd as fb
import oracle
from tests import layer_ref as ref
from tests.layer_ref import U, UB

pytestmark = pytest.mark.gpu

EPS, ALPHA = 1e-6, 0.37


def _matrix(rows, cols, dtype, seed, std=1.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    full = torch.full((rows, (-(-cols // per) + pad) * per), 77, dtype=dtype)
    full[:, :cols] = (torch.randn(rows, cols, generator=g) * std).to(dtype)
    return full.cuda()[:, :cols]


def _vector(n, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (0.8 + 0.3 * torch.randn(n + 1, generator=g)).to(dtype).cuda()[1:]  # aligned to its element only


def _np(t):
    return None if t is None else t.detach().cpu().double().numpy()


def _inputs(M, C, post, pre, gate, res, param, pad=0):
    d = {"x": _matrix(M, C, res, 1, pad=pad), "f": None, "w_post": None, "w_pre": None, "gate": None}
    if pre:
        d["w_pre"] = _vector(C, param, 2)
    if post != "none":
        d["f"] = _matrix(M, C, torch.bfloat16, 3, 2.0, pad=pad)
    if post == "norm":
        d["w_post"] = _vector(C, param, 4)
    if gate == "channel":
        d["gate"] = _vector(C, param, 5)
    elif gate == "row":
        d["gate"] = _matrix(M, C, torch.bfloat16, 6)
    return d


PARTS = [("none", True, "none")] + [p for p in itertools.product(("add", "norm"), (True, False),
                                                                 ("none", "channel", "row"))]
SIZES = [(1, 1), (3, 7), (2, 64), (5, 130), (4, 512), (7, 513), (3, 2051), (16, 7168), (2, 8192), (2, 8193), (3, 16384)]
TYPES = [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)]


def _check_forward(r, w, C, res):
    rel = 2 * (C / 2 + 8) * U
    for got, want in ((r.rstd_post, w["rstd_post"]), (r.rstd_pre, w["rstd_pre"])):
        assert (got is None) == (want is None)
        if want is not None:
            assert np.all(np.abs(_np(got) - want) <= rel * want)
    round_x = UB if res == torch.bfloat16 else U
    assert np.all(np.abs(_np(r.x) - w["x"]) <= rel * w["mag"] + round_x * np.abs(w["x"]))
    if w["n"] is None:
        return None
    scale = np.abs(w["n"]) + w["mag"] * w["rstd_pre"][:, None] * 2.0  # |w_pre| stays below 2
    tol = 2 * rel * scale
    if r.n is not None:
        assert np.all(np.abs(_np(r.n) - w["n"]) <= tol + UB * np.abs(w["n"]))
    return tol


@pytest.mark.parametrize("post,pre,gate", PARTS)
@pytest.mark.parametrize("M,C", SIZES)
@pytest.mark.parametrize("res,param", TYPES)
def test_forward(M, C, post, pre, gate, res, param):
    print(f"[layer] norm M={M} C={C} {post} {pre} {gate} {res}", flush=True)
    d = _inputs(M, C, post, pre, gate, res, param, pad=1)
    r = fb.residual_norm(alpha=ALPHA, eps=EPS, **d)
    w = ref.norm_forward(*(_np(d[k]) for k in ("x", "w_pre", "f", "w_post", "gate")), alpha=ALPHA, eps=EPS)
    assert (r.x is d["x"]) == (post == "none")
    _check_forward(r, w, C, res)


@pytest.mark.parametrize("M,C", SIZES)
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("want_n", [False, True])
def test_quantized(M, C, pow2, want_n):
    print(f"[layer] norm quantized M={M} C={C} pow2={pow2}", flush=True)
    d = _inputs(M, C, "norm", True, "channel", torch.bfloat16, torch.float32)
    r = fb.residual_norm(alpha=ALPHA, eps=EPS, quantize=True, pow2=pow2, want_n=want_n, **d)
    w = ref.norm_forward(*(_np(d[k]) for k in ("x", "w_pre", "f", "w_post", "gate")), alpha=ALPHA, eps=EPS)
    tol = _check_forward(r, w, C, torch.bfloat16)
    assert (r.n is not None) == want_n
    G = -(-C // 128)
    n = np.zeros((M, G * 128))
    t = np.zeros((M, G * 128))
    n[:, :C], t[:, :C] = w["n"], tol
    amax = np.abs(n).reshape(M, G, 128).max(2)
    slack = t.reshape(M, G, 128).max(2)
    s = _np(r.s).T
    if pow2:
        lo, hi = (np.exp2(np.ceil(np.log2(np.maximum(a, 1e-300) / 448.0))) for a in (amax - slack, amax + slack))
        assert np.all((s == lo) | (s == hi))
    else:
        assert np.all(np.abs(s * 448.0 - amax) <= slack + 2 * U * amax)
    # a code is the nearest E4M3 value: half a step of 2^-3 relative, or of 2^-9 absolute below 2^-6
    value = oracle.e4m3_decode(r.q.cpu().numpy()).astype(np.float64)
    sf = np.repeat(s, 128, axis=1)[:, :C]
    err = np.abs(value * sf - w["n"])
    assert np.all(err <= tol + sf * np.maximum(2.0 ** -4 * np.abs(w["n"]) / sf, 2.0 ** -10) * (1 + 2.0 ** -10))


def test_codes_equal_the_quantizer_on_exact_values():
    """Rows of +-2^k have the exact statistic 2^-k, so n = +-w_pre exactly (BF16
    weights): codes and scales must be those of the 1x128 quantizer, bit for bit."""
    M, C = 9, 1300
    rng = np.random.default_rng(3)
    x = torch.from_numpy(np.where(rng.random((M, C)) < 0.5, -1.0, 1.0) * np.exp2(np.arange(M) - 4)[:, None])
    x = fb.as_pitched(x.to(torch.bfloat16).cuda())
    w = (torch.randn(C, generator=torch.Generator().manual_seed(1)) * 3).to(torch.bfloat16).cuda()
    w[256:384] = 0.0  # a tile of zeros
    for pow2 in (False, True):
        r = fb.residual_norm(x, w_pre=w, eps=0.0, quantize=True, pow2=pow2)
        q, s = fb.quantize_1x128(r.n, pow2=pow2)
        assert torch.equal(r.n.float(), torch.sign(x.float()) * w.float())
        assert torch.equal(r.q, q) and torch.equal(r.s, s)


def test_in_place_and_padding():
    M, C = 11, 1003
    d = _inputs(M, C, "norm", True, "channel", torch.bfloat16, torch.float32, pad=2)
    want = fb.residual_norm(alpha=ALPHA, quantize=True, **d)
    x = d["x"]
    n, q = _matrix(M, C, torch.bfloat16, 9, pad=1), fb.empty_pitched(M, C + 40, torch.uint8)
    q.fill_(77)
    got = fb.residual_norm(alpha=ALPHA, quantize=True, x_out=x, n=n, q=q[:, :C], **d)
    assert got.x is x and torch.equal(x, want.x) and torch.equal(n, want.n) and torch.equal(q[:, :C], want.q)
    for t in (x, n):
        assert (torch.as_strided(t, (M - 1, t.stride(0) - C), (t.stride(0), 1), C) == 77).all()
    assert (q[:, C:] == 77).all()


def test_zero_rows_and_no_rows():
    C = 300
    d = _inputs(4, C, "norm", True, "none", torch.bfloat16, torch.float32)
    d["x"].zero_()
    d["f"].zero_()
    r = fb.residual_norm(eps=EPS, quantize=True, **d)
    assert not r.x.any() and not r.n.any() and not (r.q & 0x7F).any() and (r.s == 1).all()  # zeros of either sign
    assert np.allclose(_np(r.rstd_pre), 1 / np.sqrt(EPS), rtol=8 * U)
    e = {k: None if v is None else v[:0] if v.dim() == 2 else v for k, v in d.items()}
    r = fb.residual_norm(quantize=True, **e)
    assert r.x.shape == (0, C) and r.n.shape == (0, C) and r.q.shape == (0, C)
    g = fb.residual_norm_backward(e["x"], dx_out=e["x"], dn=e["f"], rstd_pre=r.rstd_pre, w_pre=d["w_pre"], f=e["f"],
                                  rstd_post=r.rstd_post, w_post=d["w_post"])
    assert g.dx.shape == (0, C) and not g.dw_pre.any() and not g.dw_post.any()


def test_a_nan_stays_in_its_row():
    d = _inputs(5, 600, "norm", True, "channel", torch.bfloat16, torch.float32)
    clean = fb.residual_norm(**d)
    d["f"][2, 17] = float("nan")
    d["x"][4, 3] = float("inf")
    r = fb.residual_norm(**d)
    for i in (0, 1, 3):
        assert torch.equal(r.n[i], clean.n[i]) and torch.equal(r.x[i], clean.x[i])
    assert torch.isnan(r.n[2]).all()


def _grads(M, C, post, pre, gate, res, param, with_dx=True):
    d = _inputs(M, C, post, pre, gate, res, param, pad=1)
    w = ref.norm_forward(*(_np(d[k]) for k in ("x", "w_pre", "f", "w_post", "gate")), alpha=ALPHA, eps=EPS)
    f32 = lambda v: None if v is None else torch.from_numpy(v).to(torch.float32).cuda()  # noqa: E731
    xo = _matrix(M, C, res, 1, pad=1)
    xo.copy_(torch.from_numpy(w["x"]).to(res))
    a = dict(dx_out=_matrix(M, C, res, 21, 0.5) if with_dx else None,
             dn=_matrix(M, C, torch.bfloat16, 22, 0.5, pad=2) if pre else None, rstd_pre=f32(w["rstd_pre"]),
             w_pre=d["w_pre"], f=d["f"], rstd_post=f32(w["rstd_post"]), w_post=d["w_post"], gate=d["gate"])
    return xo, a


@pytest.mark.parametrize("post,pre,gate", PARTS)
@pytest.mark.parametrize("M,C", SIZES + [(700, 136), (3000, 24)])
@pytest.mark.parametrize("res,param", TYPES)
def test_backward(M, C, post, pre, gate, res, param):
    print(f"[layer] norm grad M={M} C={C} {post} {pre} {gate} {res}", flush=True)
    xo, a = _grads(M, C, post, pre, gate, res, param, with_dx=not pre or (M + C) % 2 == 0)
    g = fb.residual_norm_backward(xo, alpha=ALPHA, **a)
    np_a = {k: _np(v) for k, v in a.items()}
    w = ref.norm_backward(_np(xo), alpha=ALPHA, **np_a)
    # magnitudes of the terms, for the bounds: |v|, |h| and the row's mean |v h|
    row = np.zeros((M, C)) if a["dx_out"] is None else np.abs(np_a["dx_out"])
    if pre:
        r = np_a["rstd_pre"][:, None]
        v, h = np.abs(np_a["dn"] * np_a["w_pre"]), np.abs(_np(xo)) * r
        row = row + r * (v + h * np.mean(v * h, axis=1, keepdims=True))
    rel = 2 * (C + 12) * U
    bx = rel * row
    assert np.all(np.abs(_np(g.dx) - w["dx"]) <= bx + (UB if res == torch.bfloat16 else U) * np.abs(w["dx"]))
    if pre:
        terms = np.abs(np_a["dn"] * _np(xo) * np_a["rstd_pre"][:, None]).sum(0)
        assert np.all(np.abs(_np(g.dw_pre) - w["dw_pre"]) <= 2 * (M + 4) * U * terms)
    if post == "none":
        assert g.df is None
        return
    d = ALPHA * row
    u = f = np.abs(np_a["f"])
    if post == "norm":
        f = f * np_a["rstd_post"][:, None]
        u = f * np.abs(np_a["w_post"])
    gd = 1.0 if gate == "none" else np.abs(np_a["gate"])
    if gate == "row":
        assert np.all(np.abs(_np(g.dgate) - w["dgate"]) <= 2 * rel * d * u + UB * np.abs(w["dgate"]))
    elif gate == "channel":
        assert np.all(np.abs(_np(g.dgate) - w["dgate"]) <= (2 * rel + 2 * (M + 4) * U) * (d * u).sum(0))
    d = d * gd
    if post == "norm":
        assert np.all(np.abs(_np(g.dw_post) - w["dw_post"]) <= (2 * rel + 2 * (M + 4) * U) * (d * f).sum(0))
        v = d * np.abs(np_a["w_post"])
        d = np_a["rstd_post"][:, None] * (v + f * np.mean(v * f, axis=1, keepdims=True))
    assert np.all(np.abs(_np(g.df) - w["df"]) <= 3 * rel * d + UB * np.abs(w["df"]))


# Rows that share a workgroup, in groups of 16, 32 and 64 lanes and more rows
# than groups; rows that end inside a chunk, and one channel past each limit.
ENDS = [(37, 100), (70, 129), (9001, 72), (33, 257), (41, 511), (600, 519), (5, 520), (260, 1025), (9, 4097), (9, 5001),
        (5, 8191)]


@pytest.mark.parametrize("post,pre,gate", [("none", True, "none"), ("norm", True, "channel"), ("norm", True, "row"),
                                           ("add", False, "channel")])
@pytest.mark.parametrize("M,C", ENDS)
@pytest.mark.parametrize("res,param", TYPES)
def test_row_ends_and_shared_workgroups(M, C, post, pre, gate, res, param):
    test_forward(M, C, post, pre, gate, res, param)
    if (post, gate) == ("norm", "channel"):
        test_quantized(M, C, res == torch.float32, res == torch.bfloat16)
    test_backward(M, C, post, pre, gate, res, param)


@pytest.mark.parametrize("M,C", [(50, 100), (40, 300), (300, 1025), (20, 5001), (20, 7168), (6, 9001)])
def test_backward_in_place(M, C):
    """Gradients over their own inputs, outputs' padding untouched."""
    xo, a = _grads(M, C, "norm", True, "channel", torch.bfloat16, torch.float32)
    want = fb.residual_norm_backward(xo, alpha=ALPHA, **a)
    a = {k: v if v is None or v.dim() != 2 else fb.as_pitched(v) for k, v in a.items()}
    dx, df = a["dx_out"], a["f"]
    got = fb.residual_norm_backward(xo, alpha=ALPHA, dx=dx, df=df, **a)
    assert got.dx is dx and got.df is df
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("C", [64, 100, 1025, 7168])
def test_backward_without_a_norm_copies(C):
    d = _matrix(9, C, torch.bfloat16, 3)
    out = _matrix(9, C, torch.bfloat16, 4)
    g = fb.residual_norm_backward(d, dx_out=d, dx=out)
    assert g.dx is out and torch.equal(out, d) and g.df is None and g.dw_pre is None


def test_backward_twice_is_the_same():
    xo, a = _grads(2000, 264, "norm", True, "channel", torch.bfloat16, torch.float32)
    one, two = (fb.residual_norm_backward(xo, alpha=ALPHA, **a) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(one, two))


def test_gradient_by_differences():
    """Against central differences of the 64-bit forward: loss = <x', A> + <n, B>."""
    M, C = 3, 40
    d = _inputs(M, C, "norm", True, "channel", torch.float32, torch.float32)
    d["f"] = _matrix(M, C, torch.bfloat16, 3)
    A, B = _matrix(M, C, torch.float32, 31), _matrix(M, C, torch.bfloat16, 32)
    r = fb.residual_norm(alpha=ALPHA, eps=EPS, **d)
    g = fb.residual_norm_backward(r.x, dx_out=A, dn=B, rstd_pre=r.rstd_pre, w_pre=d["w_pre"], f=d["f"],
                                  rstd_post=r.rstd_post, w_post=d["w_post"], gate=d["gate"], alpha=ALPHA)
    p = {k: _np(v) for k, v in d.items()}

    def loss(q):
        w = ref.norm_forward(q["x"], q["w_pre"], q["f"], q["w_post"], q["gate"], alpha=ALPHA, eps=EPS)
        return float((w["x"] * _np(A)).sum() + (w["n"] * _np(B)).sum())

    h = 2.0 ** -12
    rng = np.random.default_rng(5)
    size = float(np.abs(_np(A)).sum() + np.abs(_np(B)).sum())  # of the loss and its derivatives, entries of order one
    for name, got in (("x", g.dx), ("f", g.df), ("w_pre", g.dw_pre), ("w_post", g.dw_post), ("gate", g.dgate)):
        G = _np(got)
        for _ in range(12):
            i = tuple(int(rng.integers(n)) for n in G.shape)
            lo, hi = dict(p), dict(p)
            lo[name], hi[name] = p[name].copy(), p[name].copy()
            lo[name][i] -= h
            hi[name][i] += h
            d_ = (loss(hi) - loss(lo)) / (2 * h)
            # h^2 times a third derivative, FP32 sums of 2 C terms, df's rounding to BF16
            assert abs(G[i] - d_) <= size * (h * h + 4 * C * U) + (UB * abs(d_) if name == "f" else 0), (name, i)
