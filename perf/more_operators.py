"""Workloads of the gated feed-forward block in FP8 and of the optimizer step.

* ``gated``       gate and up projection in one product with the activation,
                  h = act(x Wg) * (x Wu), for one weight matrix or for the
                  experts of a mixture (rows ordered by expert).
* ``ffn``         the same with h quantized to 1x128 E4M3 on store, and the down
                  projection that reads it.
* ``gated_grad``  gradient of the block's input side: the down projection's
                  input gradient and the activation's in one product; with
                  ``dx`` quantized on store for the up projection's.
* ``adamw``       one AdamW step over many tensors, gradients clipped by a given
                  norm, moments in FP32, BF16 or E4M3 with a scale for 128 values.

``run`` is the plain form (elementary torch operations in 32 bits, rounded once
at the end) unless ``own`` is set: then it calls the package's entry points.
Sizes follow the package's mixture-of-experts workload: 8192 tokens, 256
experts, 8 of them per token, hidden size 7168, expert width 2048.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
LR, BETA1, BETA2, EPS, DECAY, STEP = 3e-4, 0.9, 0.95, 1e-8, 0.1, 20
CLIP_EPS = 1e-6


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 16 sequences through a shared expert
        dict(name="gated_decode", kind="gated", T=16, top=0, E=0, K=7168, H=2048, act="silu", t=False, pow2=False,
             u=False),
        # a short prompt, odd row count, weights stored transposed, power-of-two scales, kept for the gradient
        dict(name="gated_odd", kind="gated", T=777, top=0, E=0, K=2048, H=1408, act="gelu", t=True, pow2=True, u=True),
        # decode: 16 tokens to 8 of 256 experts each, most experts with one row or none
        dict(name="gated_experts_decode", kind="gated", T=16, top=8, E=256, K=7168, H=2048, act="silu", t=False,
             pow2=False, u=False),
        # prompt of 8192 tokens through the shared expert, FP8 between the projections
        dict(name="ffn_prompt", kind="ffn", T=8192, top=0, E=0, K=7168, H=2048, act="silu", t=False, pow2=False,
             u=False),
        # training forward of the experts
        dict(name="ffn_experts_train", kind="ffn", T=8192, top=8, E=256, K=7168, H=2048, act="silu", t=False,
             pow2=False, u=True),
        # gradient at an odd row count
        dict(name="grad_odd", kind="gated_grad", T=777, top=0, E=0, K=2048, H=1408, act="gelu", t=False, pow2=True,
             dx=False),
        # training backward of the shared expert
        dict(name="grad_shared", kind="gated_grad", T=8192, top=0, E=0, K=7168, H=2048, act="silu", t=True, pow2=False,
             dx=False),
        # training backward of the experts
        dict(name="grad_experts_train", kind="gated_grad", T=8192, top=8, E=256, K=7168, H=2048, act="silu", t=True,
             pow2=False, dx=True),
        # the small parameters of a model: biases, norms, routers
        dict(name="adamw_small", kind="adamw", n=200, total=1200007, param="f32", grad="mixed", state="f32", copy=False,
             random=False),
        # parameters held in BF16 with BF16 moments, rounded at random
        dict(name="adamw_bf16", kind="adamw", n=40, total=60000011, param="bf16", grad="bf16", state="bf16", copy=False,
             random=True),
        # 64 experts' down projections: FP32 weights and moments, BF16 copies for the products
        dict(name="adamw_experts_f32", kind="adamw", n=64, total=64 * 2048 * 7168, param="f32", grad="f32", state="f32",
             copy=True, random=False),
        # the same with moments in 8 bits
        dict(name="adamw_experts_e4m3", kind="adamw", n=64, total=64 * 2048 * 7168, param="f32", grad="f32",
             state="e4m3", copy=True, random=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["gated", "ffn", "gated_grad", "adamw"])
    if kind == "adamw":
        n = _log(rng, 1, 400)
        return dict(kind=kind, n=n, total=_log(rng, 1000 + n, 200000000), param=rng.choice(["bf16", "f32"]),
                    grad=rng.choice(["bf16", "f32", "mixed"]), state=rng.choice(["f32", "bf16", "e4m3"]),
                    copy=rng.choice([True, False]), random=rng.choice([True, False]))
    c = dict(kind=kind, T=_log(rng, 1, 8192), top=0, E=0, K=128 * _log(rng, 1, 56), H=128 * _log(rng, 1, 16),
             act=rng.choice(["silu", "silu", "gelu"]), t=rng.choice([True, False]), pow2=rng.choice([True, False]))
    if rng.random() < 0.5:
        c.update(T=_log(rng, 1, 2048), top=rng.randint(1, 8), E=_log(rng, 8, 64))
    if kind == "gated_grad":
        return dict(c, dx=rng.choice([True, False]))
    return dict(c, u=rng.choice([True, False]))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _dt(s):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[s]


def _codes(g, shape, std):
    """E4M3 codes of normal values, a matrix at a time."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for m in out.view(-1, *shape[-2:]):
        v = torch.randn(shape[-2:], generator=g, device="cuda").mul_(std).clamp_(-E4M3_MAX, E4M3_MAX)
        m.copy_(v.to(torch.float8_e4m3fn).view(torch.uint8))
    return out


def _scales(g, shape, mean, pow2):
    s = mean * (0.6 + 0.8 * torch.rand(shape, generator=g, device="cuda"))
    return torch.exp2(torch.round(torch.log2(s))) if pow2 else s


def _activations(g, rows, cols, rms, pow2):
    """Codes [rows][cols] and scales [cols/128][rows] of values of that size: a
    tile's largest of 128 values is about 2.8 times their size."""
    return _codes(g, (rows, cols), E4M3_MAX / 2.8), _scales(g, (cols // 128, rows), rms * 2.8 / E4M3_MAX, pow2)


def _weights(g, c, rows, cols, fan_in):
    """Codes and 128x128 scales of a matrix, or of one for each expert."""
    lead = (c["E"],) if c["E"] else ()
    q = _codes(g, (*lead, rows, cols), E4M3_MAX / 4.5)
    return q, _scales(g, (*lead, rows // 128, cols // 128), fan_in ** -0.5 * 4.5 / E4M3_MAX, c["pow2"])


def _sizes(c):
    """n tensor sizes from 1 element up that add up to `total`."""
    if c["total"] % c["n"] == 0 and c["param"] == "f32" and c["grad"] == "f32":
        return [c["total"] // c["n"]] * c["n"]
    share = np.random.RandomState(c["n"]).lognormal(0.0, 2.0, c["n"])
    size = 1 + np.floor(share / share.sum() * (c["total"] - c["n"])).astype(np.int64)
    size[int(np.argmax(size))] += c["total"] - int(size.sum())
    return [int(v) for v in size]


def _prepare_adamw(c, g):
    sizes = _sizes(c)
    total = c["total"]

    def flat(t):
        return torch.empty(total, dtype=t, device="cuda")

    s = {"case": c, "sizes": sizes, "p": flat(_dt(c["param"])), "plan": {}}
    s["p"].copy_(torch.randn(total, generator=g, device="cuda") * 0.02)
    s["params"] = list(torch.split(s["p"], sizes))
    kinds = [{"bf16": torch.bfloat16, "f32": torch.float32}.get(c["grad"]) or
             (torch.bfloat16 if i % 2 else torch.float32) for i in range(len(sizes))]
    s["grads"] = [(torch.randn(n, generator=g, device="cuda") * 1e-3).to(t) for n, t in zip(sizes, kinds)]
    s["decay"] = [DECAY if i % 3 else 0.0 for i in range(len(sizes))]  # norms and biases have none
    s["norm"] = torch.tensor(1e-3 * math.sqrt(total), device="cuda") * (0.9 + 0.2 * torch.rand((), generator=g, device="cuda"))
    s["max_norm"] = 0.5e-3 * math.sqrt(total)
    s["seed"] = int(torch.randint(0, 2 ** 31 - 1, (), generator=g, device="cuda")) if c["random"] else None
    if c["copy"]:
        s["c"] = flat(torch.bfloat16)
        s["copies"] = list(torch.split(s["c"], sizes))
    if c["state"] != "e4m3":
        t = _dt(c["state"])
        s["m"], s["v"] = flat(t), flat(t)
        s["m"].copy_(torch.randn(total, generator=g, device="cuda") * 3e-4)
        s["v"].copy_(torch.randn(total, generator=g, device="cuda").square_() * 1e-6 + 1e-8)
        s["ms"], s["vs"] = list(torch.split(s["m"], sizes)), list(torch.split(s["v"], sizes))
        return s
    groups = [-(-n // 128) for n in sizes]  # a tensor's codes fill whole groups of 128
    G = sum(groups)
    s["m"] = _codes(g, (1, G * 128), E4M3_MAX / 2.8).view(-1)
    s["v"] = _codes(g, (1, G * 128), E4M3_MAX / 2.8).view(-1) & 0x7F
    if G * 128 != total:  # nothing behind a tensor's end
        for q in (s["m"], s["v"]):
            at = 0
            for n, k in zip(sizes, groups):
                q[at + n:at + 128 * k] = 0
                at += 128 * k
    s["m_scale"] = _scales(g, (G,), 3e-4 * 2.8 / E4M3_MAX, False)
    s["v_scale"] = _scales(g, (G,), 1e-3 * 2.8 / E4M3_MAX, False)
    s["ms"] = [t[:n] for t, n in zip(torch.split(s["m"], [128 * k for k in groups]), sizes)]
    s["vs"] = [t[:n] for t, n in zip(torch.split(s["v"], [128 * k for k in groups]), sizes)]
    s["m_scales"], s["v_scales"] = list(torch.split(s["m_scale"], groups)), list(torch.split(s["v_scale"], groups))
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    if c["kind"] == "adamw":
        return _prepare_adamw(c, g)
    s = {"case": c}
    P, K, H = c["T"] * max(c["top"], 1), c["K"], c["H"]
    if c["E"]:  # rows of every expert, from a top-k over skewed scores
        bias = torch.randn(c["E"], generator=g, device="cuda") * 0.5
        ids = torch.topk(torch.sigmoid(torch.randn(c["T"], c["E"], generator=g, device="cuda") + bias), c["top"], 1)[1]
        counts = torch.bincount(ids.view(-1), minlength=c["E"])
        s["offsets"] = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)]).to(torch.int32)
        s["bounds"] = s["offsets"].tolist()  # the plain form's loop over the experts
    if c["kind"] != "gated_grad":
        s["x"], s["sx"] = _activations(g, P, K, 1.0, c["pow2"])
        s["up"], s["s_up"] = _weights(g, c, *((2 * H, K) if c["t"] else (K, 2 * H)), K)
        if c["kind"] == "ffn":
            s["down"], s["s_down"] = _weights(g, c, H, K, H)
        return s
    s["u"] = torch.randn(P, 2 * H, generator=g, device="cuda").to(torch.bfloat16)
    s["do"], s["s_do"] = _activations(g, P, K, 1e-3, c["pow2"])
    s["down"], s["s_down"] = _weights(g, c, *((H, K) if c["t"] else (K, H)), H)
    if c["dx"]:
        s["up"], s["s_up"] = _weights(g, c, K, 2 * H, K)
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _value(q):
    return q.view(torch.float8_e4m3fn).float()


def _rows_value(q, s):
    """The values of codes with a scale for a row's 128 columns, s [cols/128][rows]."""
    M, C = q.shape
    return (_value(q).view(M, C // 128, 128) * s.t()[:, :, None]).view(M, C)


def _block_value(q, s):
    """The values of codes with a scale for 128x128 of them."""
    R, C = q.shape
    return (_value(q).view(R // 128, 128, C // 128, 128) * s[:, None, :, None]).view(R, C)


def _product(s, x, q, scales, t):
    """x times the weights, expert by expert where there are several."""
    def times(rows, w, ws):
        w = _block_value(w, ws)
        return rows @ (w.t() if t else w)

    if "bounds" not in s:
        return times(x, q, scales)
    b = s["bounds"]
    return torch.cat([times(x[lo:hi], q[e], scales[e]) for e, (lo, hi) in enumerate(zip(b[:-1], b[1:])) if hi > lo])


def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _arg(g, act):
    """act(g) = g sigmoid(z): g itself, or the cubic of the tanh form of the GELU; and dz/dg."""
    if act == "silu":
        return g, torch.ones_like(g)
    k = math.sqrt(8.0 / math.pi)
    return k * (g + 0.044715 * g * g * g), k * (1.0 + 3.0 * 0.044715 * g * g)


def _quantize(h, pow2):
    """h [M][C] (C a multiple of 128) as stored in BF16: codes and scales of its 1x128 tiles."""
    M, C = h.shape
    t = h.to(torch.bfloat16).float().view(M, C // 128, 128)
    top = t.abs().amax(2)
    sc = top / E4M3_MAX
    if pow2:
        m, e = torch.frexp(sc)
        sc = torch.ldexp(torch.ones_like(sc), torch.where(m == 0.5, e - 1, e))
    sc = torch.where(top == 0, torch.ones_like(sc), sc)
    q = (t / sc[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(M, C).view(torch.uint8), sc.t()


def _plain_gated(s, c):
    H = c["H"]
    u = _product(s, _rows_value(s["x"], s["sx"]), s["up"], s["s_up"], c["t"])
    g, v = u[:, :H], u[:, H:]
    h = g * _sigmoid(_arg(g, c["act"])[0]) * v
    out = {"u": u.to(torch.bfloat16)} if c["u"] else {}
    if c["kind"] == "gated":
        return dict(out, h=h.to(torch.bfloat16))
    y = _product(s, _rows_value(*_quantize(h, c["pow2"])), s["down"], s["s_down"], False)
    return dict(out, y=y.to(torch.bfloat16))


def _plain_gated_grad(s, c):
    H = c["H"]
    dh = _product(s, _rows_value(s["do"], s["s_do"]), s["down"], s["s_down"], c["t"])
    g, v = s["u"][:, :H].float(), s["u"][:, H:].float()
    z, dz = _arg(g, c["act"])
    p = _sigmoid(z)
    a = g * p
    du = torch.cat([dh * v * (p + a * (1.0 - p) * dz), dh * a], 1)
    out = {"du": du.to(torch.bfloat16), "h": (a * v).to(torch.bfloat16)}
    if c["dx"]:
        out["dx"] = _product(s, _rows_value(*_quantize(du, c["pow2"])), s["up"], s["s_up"], True).to(torch.bfloat16)
    return out


def _hash(seed, n):
    """32 random bits for each of n elements: a mix of their index and the seed."""
    i = torch.arange(n, dtype=torch.int64, device="cuda")
    h = ((i * 0x9E3779B1) ^ (i >> 32)) + seed & 0xFFFFFFFF
    h = (h ^ (h >> 16)) * 0x85EBCA6B & 0xFFFFFFFF
    h = (h ^ (h >> 13)) * 0xC2B2AE35 & 0xFFFFFFFF
    return h ^ (h >> 16)


def _drop(x, bits, r):
    """x (FP32) without its lowest bits, after the random bits r were added there."""
    w = x.view(torch.int32).long() & 0xFFFFFFFF
    w = (w + r) >> bits << bits & 0xFFFFFFFF
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).view(torch.float32)


def _to_bf16(x, r):
    return x.to(torch.bfloat16) if r is None else _drop(x, 16, r).to(torch.bfloat16)


def _to_e4m3(x, r, floor):
    """Codes of 128 values each under one scale; floor: what is not zero keeps at least the smallest code."""
    n = x.numel()
    t = torch.nn.functional.pad(x, (0, -n % 128)).view(-1, 128)
    top = t.abs().amax(1)
    sc = torch.where(top == 0, torch.ones_like(top), top / E4M3_MAX)
    y = (t / sc[:, None]).view(-1)[:n]
    a = y.abs().clamp(max=E4M3_MAX)
    if r is not None:  # below 2^-6 codes are 2^-9 apart, as they are from there to 2^-5
        a = torch.where(a < 2.0 ** -6, _drop(a + 2.0 ** -6, 20, r << 4) - 2.0 ** -6, _drop(a, 20, r << 4))
    q = a.to(torch.float8_e4m3fn).float()
    if floor:
        q = torch.where((x > 0) & (q == 0), torch.full_like(q, 2.0 ** -9), q)
    return torch.copysign(q, y).to(torch.float8_e4m3fn).view(torch.uint8), sc


def _plain_adamw_one(s, c, i, clip):
    p, n = s["params"][i], s["sizes"][i]
    w, g = p.float(), s["grads"][i].float() * clip
    seed = None if s["seed"] is None else (s["seed"] + i * 0x27D4EB2F) & 0xFFFFFFFF
    rm = rv = rp = None
    if seed is not None:
        r = _hash(seed, n)
        rm, rv = r & 0xFFFF, r >> 16
        rp = _hash(seed ^ 0x5BD1E995, n) & 0xFFFF
    if c["state"] == "e4m3":
        mq, vq, msc, vsc = s["ms"][i], s["vs"][i], s["m_scales"][i], s["v_scales"][i]
        m = _value(mq) * msc.repeat_interleave(128)[:n]
        v = (_value(vq) * vsc.repeat_interleave(128)[:n]).square()
    else:
        m, v = s["ms"][i].float(), s["vs"][i].float()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    step = LR / (1 - BETA1 ** STEP) * m / (torch.sqrt(v) / math.sqrt(1 - BETA2 ** STEP) + EPS)
    w = w * (1 - LR * s["decay"][i]) - step
    if c["state"] == "f32":
        s["ms"][i].copy_(m)
        s["vs"][i].copy_(v)
    elif c["state"] == "bf16":
        s["ms"][i].copy_(_to_bf16(m, rm))
        s["vs"][i].copy_(_to_bf16(v, rv))
    else:
        for q, sc, got in ((mq, msc, _to_e4m3(m, rm, False)), (vq, vsc, _to_e4m3(torch.sqrt(v), rv, True))):
            q.copy_(got[0])
            sc.copy_(got[1])
    if c["param"] == "f32":
        p.copy_(w)
    else:
        p.copy_(_to_bf16(w, rp))
    if c["copy"]:
        s["copies"][i].copy_(w)


def _adamw_out(s, c):
    out = {"p": s["p"]}
    if c["copy"]:
        out["copy"] = s["c"]
    if c["state"] != "e4m3":
        return dict(out, m=s["m"], v=s["v"])
    return dict(out, m=s["m"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn), m_scale=s["m_scale"],
                v_scale=s["v_scale"])


def _plain(s):
    c = s["case"]
    if c["kind"] == "adamw":
        clip = (s["max_norm"] / (s["norm"] + CLIP_EPS)).clamp(max=1.0)
        [_plain_adamw_one(s, c, i, clip) for i in range(len(s["sizes"]))]
        return _adamw_out(s, c)
    return _plain_gated_grad(s, c) if c["kind"] == "gated_grad" else _plain_gated(s, c)


# --------------------------------------------------------------------------
# the package's calls
# --------------------------------------------------------------------------
def _called(s):
    import fp8_fine_grained_quantize_amd as fb

    c = s["case"]
    if c["kind"] == "adamw":
        if "table" not in s["plan"]:
            state = fb.AdamWState(s["params"], s["ms"], s["vs"], m_scales=s.get("m_scales"), v_scales=s.get("v_scales"),
                                  copies=s.get("copies"), decay=s["decay"])
            s["plan"]["table"] = fb.adamw_table(state, s["grads"])
        fb.adamw_step(s["plan"]["table"], LR, STEP, beta1=BETA1, beta2=BETA2, eps=EPS, norm=s["norm"],
                      max_norm=s["max_norm"], clip_eps=CLIP_EPS, seed=s["seed"])
        return _adamw_out(s, c)
    kept = dict(act=c["act"], pow2_scales=c["pow2"])
    plain = dict(pow2_scales=c["pow2"], out_dtype=torch.bfloat16)
    by = fb.OP_T if c["t"] else fb.OP_N
    experts = "offsets" in s
    if c["kind"] != "gated_grad":
        kept.update(opB=by, want_u=c["u"])
        if c["kind"] == "ffn":
            kept.update(quantize=True, pow2=c["pow2"], want_h=False)
        if experts:
            r = fb.grouped_gated_gemm_fp8_blockscaled(s["offsets"], s["x"], s["sx"], s["up"], s["s_up"], **kept)
        else:
            r = fb.gated_gemm_fp8_blockscaled(s["x"], s["sx"], s["up"], s["s_up"], **kept)
        out = {"u": r.u} if c["u"] else {}
        if c["kind"] == "gated":
            return dict(out, h=r.h)
        if experts:
            return dict(out, y=fb.grouped_gemm_fp8_blockscaled(s["offsets"], r.q, r.s, s["down"], s["s_down"], **plain))
        return dict(out, y=fb.gemm_fp8_blockscaled(r.q, r.s, s["down"], s["s_down"], **plain))
    kept.update(opB=by, quantize=c["dx"], pow2=c["pow2"])
    if experts:
        r = fb.grouped_gated_gemm_backward_fp8_blockscaled(s["offsets"], s["do"], s["s_do"], s["down"], s["s_down"],
                                                           s["u"], **kept)
    else:
        r = fb.gated_gemm_backward_fp8_blockscaled(s["do"], s["s_do"], s["down"], s["s_down"], s["u"], **kept)
    out = {"du": r.du, "h": r.h}
    if c["dx"] and experts:
        out["dx"] = fb.grouped_gemm_fp8_blockscaled(s["offsets"], r.q, r.s, s["up"], s["s_up"], opB=fb.OP_T, **plain)
    elif c["dx"]:
        out["dx"] = fb.gemm_fp8_blockscaled(r.q, r.s, s["up"], s["s_up"], opB=fb.OP_T, **plain)
    return out


def run(state):
    return _called(state) if own else _plain(state)


# --------------------------------------------------------------------------
# what a pass cannot do without, each input read once, each output written once
# --------------------------------------------------------------------------
def work(case):
    c = case
    if c["kind"] == "adamw":
        n = c["total"]
        at = {"f32": 4.0, "bf16": 2.0}
        if c["grad"] == "mixed":
            got = sum(k * (2 if i % 2 else 4) for i, k in enumerate(_sizes(c)))
        else:
            got = n * at[c["grad"]]
        st = n * (1 + 4 / 128) if c["state"] == "e4m3" else n * at[c["state"]]
        return {"bytes": got + 2 * n * at[c["param"]] + 4 * st + (2 * n if c["copy"] else 0), "flops": 15 * n}
    P, K, H, E = c["T"] * max(c["top"], 1), c["K"], c["H"], c["E"]
    used = E * (1 - (1 - 1 / E) ** P) if E else 1  # experts that have a row at all
    rows = P * (K + K / 32)
    up, down = used * 2 * H * K, used * H * K
    if c["kind"] == "gated_grad":
        b = rows + down + P * H * (4 + 4 + 2)
        f = 2 * P * K * H
        return {"bytes": b + (up + 2 * P * K if c["dx"] else 0), "flops": f + (2 * f if c["dx"] else 0)}
    b = rows + up + (4 * P * H if c["u"] else 0)
    f = 4 * P * K * H
    if c["kind"] == "gated":
        return {"bytes": b + 2 * P * H, "flops": f}
    return {"bytes": b + down + 2 * P * K, "flops": f + 2 * P * K * H}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_codes(q, *spread):
    """Values of codes; spread: (scales, how many codes one stands for along either axis)."""
    s, r, k = spread
    v = q.view(torch.float8_e4m3fn).double()
    return v * torch.kron(s.double().contiguous(), torch.ones(r, k, dtype=torch.float64, device=q.device))


def _exact_product(s, x, q, scales, t):
    K = x.shape[1]
    N = q.shape[-2] if t else q.shape[-1]
    y = torch.zeros(x.shape[0], N, dtype=torch.float64, device="cuda")
    b = s.get("bounds", [0, x.shape[0]])
    q, scales = q.view(-1, *q.shape[-2:]), scales.view(-1, *scales.shape[-2:])
    for e in range(len(b) - 1):
        if b[e] == b[e + 1]:
            continue
        w = _exact_codes(q[e], scales[e], 128, 128)
        assert (w.shape[1] if t else w.shape[0]) == K
        y[b[e]:b[e + 1]] = torch.mm(x[b[e]:b[e + 1]], w.T if t else w)
    return y


def _exact_act(g, act):
    """The activation and its derivative, by tanh: sigmoid(z) = (1 + tanh(z / 2)) / 2."""
    if act == "silu":
        th, dz = torch.tanh(g / 2), 1.0
    else:
        th, dz = torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)), math.sqrt(8 / math.pi) * (1 + 0.134145 * g ** 2)
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.25 * g * (1 - th) * (1 + th) * dz


def _exact_rounded(h, pow2):
    """The values that h stands for after its tiles were rounded to BF16 and to codes."""
    h = h.to(torch.bfloat16).double()
    for a in range(0, h.shape[1], 128):
        t = h[:, a:a + 128]
        m = t.abs().max(1, keepdim=True).values
        sc = torch.exp2(torch.ceil(torch.log2(m / E4M3_MAX))) if pow2 else m / E4M3_MAX
        sc = torch.where(m == 0, torch.ones_like(sc), sc)
        h[:, a:a + 128] = (t / sc).to(torch.float8_e4m3fn).double() * sc
    return h


def _exact_adamw(s, c):
    out = _adamw_out(s, c)
    got = {k: torch.zeros(v.numel(), dtype=torch.float64, device="cuda") for k, v in out.items()}
    scale = min(1.0, s["max_norm"] / (float(s["norm"]) + CLIP_EPS))
    at = code = group = 0
    for i, n in enumerate(s["sizes"]):
        g = s["grads"][i].double() * scale
        k = -(-n // 128)
        if c["state"] == "e4m3":
            spread = torch.arange(n, device="cuda") // 128
            m = s["ms"][i].view(torch.float8_e4m3fn).double() * s["m_scales"][i].double()[spread]
            root = s["vs"][i].view(torch.float8_e4m3fn).double() * s["v_scales"][i].double()[spread]
            v = root * root
        else:
            m, v = s["ms"][i].double(), s["vs"][i].double()
        m = m + (1 - BETA1) * (g - m)
        v = v + (1 - BETA2) * (g * g - v)
        p = s["params"][i].double()
        p = p - LR * s["decay"][i] * p - LR * (m / (1 - BETA1 ** STEP)) / (torch.sqrt(v / (1 - BETA2 ** STEP)) + EPS)
        got["p"][at:at + n] = p
        if c["copy"]:
            got["copy"][at:at + n] = p
        if c["state"] == "e4m3":
            for name, x in (("m", m), ("v", torch.sqrt(v))):
                x = torch.cat([x, x.new_zeros(128 * k - n)]).view(k, 128)
                top = x.abs().max(1).values
                sc = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
                got[name + "_scale"][group:group + k] = sc
                got[name][code:code + 128 * k] = (x / sc[:, None]).view(-1)  # before it is rounded to a code
        else:
            got["m"][at:at + n], got["v"][at:at + n] = m, v
        at, code, group = at + n, code + 128 * k, group + k
    return got


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["kind"] == "adamw":
        return _exact_adamw(s, c)
    H = c["H"]
    if c["kind"] != "gated_grad":
        x = _exact_codes(s["x"], s["sx"].T, 1, 128)
        u = _exact_product(s, x, s["up"], s["s_up"], c["t"])
        h = _exact_act(u[:, :H], c["act"])[0] * u[:, H:]
        out = {"u": u} if c["u"] else {}
        if c["kind"] == "gated":
            return dict(out, h=h)
        return dict(out, y=_exact_product(s, _exact_rounded(h, c["pow2"]), s["down"], s["s_down"], False))
    dh = _exact_product(s, _exact_codes(s["do"], s["s_do"].T, 1, 128), s["down"], s["s_down"], c["t"])
    u = s["u"].double()
    a, da = _exact_act(u[:, :H], c["act"])
    du = torch.empty_like(u)
    du[:, :H], du[:, H:] = dh * u[:, H:] * da, dh * a
    out = {"du": du, "h": a * u[:, H:]}
    if c["dx"]:
        out["dx"] = _exact_product(s, _exact_rounded(du, c["pow2"]), s["up"], s["s_up"], True)
    return out
