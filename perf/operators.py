"""Workloads of the operators around the FP8 GEMMs of a mixture-of-experts layer.

* ``sort``          (token, slot) pairs sorted by expert: offsets and both maps.
* ``dispatch``      token rows copied into expert order, in BF16 or as E4M3
                    codes with their 1x128 scales.
* ``combine``       expert rows back to tokens, with the router's weights; with
                    no weights it is the gradient of ``dispatch``.
* ``combine_grad``  its gradient: expert rows and weights.
* ``clip``          global gradient norm over many tensors, and clipping.
* ``norm``          the norm after a block with its gate and residual scale,
                    the residual sum, and the norm before the next block,
                    optionally quantized to 1x128 E4M3.
* ``norm_grad``     its gradient.

``run`` is the plain form (elementary torch operations in 32 bits, rounded once
at the end) unless ``own`` is set: then it calls the package's entry points.
Sizes follow the package's mixture-of-experts workload: 8192 tokens, 256
experts, 8 of them per token, hidden size 7168, expert width 2048.
"""
import math

import numpy as np
import torch

own = False

EPS_NORM = 1e-6
EPS_CLIP = 1e-6
ALPHA = 0.5
E4M3_MAX = 448.0


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 16 sequences: latency of the smallest sort
        dict(name="sort_decode", kind="sort", T=16, K=8, E=256, drop=0.0, ids="int64"),
        # a training micro-batch, some pairs masked (padding tokens)
        dict(name="sort_train", kind="sort", T=8192, K=8, E=256, drop=0.03, ids="int64"),
        # quantized activations sent to their experts (training forward)
        dict(name="dispatch_fp8_train", kind="dispatch", T=8192, K=8, E=256, C=7168, drop=0.0, type="fp8"),
        # BF16 rows of a short prompt with an odd hidden size, two experts per token
        dict(name="dispatch_bf16_odd", kind="dispatch", T=777, K=2, E=64, C=2051, drop=0.05, type="bf16"),
        # decode: the experts' rows of 16 tokens back to them
        dict(name="combine_decode", kind="combine", T=16, K=8, E=256, C=7168, drop=0.0, rows="bf16", out="bf16",
             weighted=True),
        # training forward: FP32 rows as the grouped GEMM writes them by default
        dict(name="combine_train", kind="combine", T=8192, K=8, E=256, C=7168, drop=0.0, rows="f32", out="bf16",
             weighted=True),
        # training backward: gradient rows and router-weight gradients
        dict(name="combine_grad_train", kind="combine_grad", T=8192, K=8, E=256, C=7168, drop=0.0, rows="bf16",
             out="bf16"),
        # the small parameters of a model: biases, norms, routers
        dict(name="clip_small", kind="clip", n=200, total=1200007, types="mixed", out="f32", clips=True),
        # 64 experts' down-projection weight gradients
        dict(name="clip_experts", kind="clip", n=64, total=64 * 2048 * 7168, types="f32", out="f32", clips=True),
        # decode: residual sum and the next block's norm, quantized for its GEMM
        dict(name="norm_decode", kind="norm", M=16, C=7168, post="norm", pre=True, gate="channel", res="bf16",
             param="f32", quant="pow2"),
        # training forward between two blocks
        dict(name="norm_train", kind="norm", M=8192, C=7168, post="norm", pre=True, gate="channel", res="bf16",
             param="f32", quant="fp32"),
        # training backward between two blocks
        dict(name="norm_grad_train", kind="norm_grad", M=8192, C=7168, post="norm", pre=True, gate="channel",
             res="bf16", param="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["sort", "dispatch", "combine", "combine_grad", "clip", "norm", "norm_grad"])
    if kind in ("sort", "dispatch", "combine", "combine_grad"):
        c = dict(kind=kind, T=_log(rng, 1, 8192), K=rng.randint(1, 8), E=_log(rng, 8, 384),
                 drop=rng.choice([0.0, 0.0, 0.02, 0.3]))
        if kind == "sort":
            return dict(c, T=_log(rng, 1, 32768), ids=rng.choice(["int32", "int64"]))
        c["C"] = _log(rng, 64, 7168)
        if kind == "dispatch":
            return dict(c, type=rng.choice(["bf16", "fp8"]))
        c["rows"], c["out"] = rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"])
        if kind == "combine":
            return dict(c, weighted=rng.choice([True, True, False]))
        return c
    if kind == "clip":
        n = _log(rng, 1, 400)
        return dict(kind=kind, n=n, total=_log(rng, 1000 + n, 200000000), types=rng.choice(["bf16", "f32", "mixed"]),
                    out=rng.choice(["bf16", "f32"]), clips=rng.choice([True, True, False]))
    c = dict(kind=kind, M=_log(rng, 1, 8192), C=_log(rng, 64, 8192), post=rng.choice(["norm", "norm", "add", "none"]),
             pre=True, gate="none", res=rng.choice(["bf16", "f32"]), param=rng.choice(["bf16", "f32"]))
    if c["post"] != "none":
        c["pre"] = rng.choice([True, True, False])
        c["gate"] = rng.choice(["none", "channel", "row"])
    if kind == "norm":
        c["quant"] = rng.choice(["none", "fp32", "pow2"]) if c["pre"] else "none"
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _dt(s):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[s]


def _pitched(rows, cols, dtype):
    """[rows][cols] on the GPU whose rows lie a multiple of 16 bytes apart."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.empty(rows, -(-cols // per) * per, dtype=dtype, device="cuda")[:, :cols]


def _randn(g, rows, cols, dtype, std=1.0):
    t = _pitched(rows, cols, dtype)
    t.copy_(torch.randn(rows, cols, generator=g, device="cuda") * std)
    return t


def _routing(c, g):
    """Top-K experts of every token (skewed by an expert bias), the router's
    weights, and the maps that sorting the pairs by expert gives."""
    T, K, E = c["T"], c["K"], c["E"]
    bias = torch.randn(E, generator=g, device="cuda") * 0.5
    aff = torch.sigmoid(torch.randn(T, E, generator=g, device="cuda") + bias)
    top = torch.topk(aff, K, dim=1)
    w = top.values / top.values.sum(1, keepdim=True)
    ids = top.indices
    if c["drop"]:
        ids = torch.where(torch.rand(T, K, generator=g, device="cuda") < c["drop"], torch.full_like(ids, -1), ids)
    return ids, w.contiguous()


def _sizes(c):
    """n tensor sizes from 1 element up that add up to `total`."""
    if c["total"] % c["n"] == 0 and c["types"] == "f32":
        return [c["total"] // c["n"]] * c["n"]
    share = np.random.RandomState(c["n"]).lognormal(0.0, 2.0, c["n"])
    size = 1 + np.floor(share / share.sum() * (c["total"] - c["n"])).astype(np.int64)
    size[int(np.argmax(size))] += c["total"] - int(size.sum())
    return [int(v) for v in size]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    kind = c["kind"]
    s = {"case": c}
    if kind in ("sort", "dispatch", "combine", "combine_grad"):
        ids, w = _routing(c, g)
        if kind == "sort":
            s["ids"] = ids.to(torch.int32) if c["ids"] == "int32" else ids
            return s
        offsets, row_of, slot_of = _plain_sort(ids, c["E"])
        s.update(row_of=row_of, slot_of=slot_of)
        P, C = c["T"] * c["K"], c["C"]
        if kind == "dispatch":
            if c["type"] == "bf16":
                s["x"] = _randn(g, c["T"], C, torch.bfloat16)
            else:
                q = _pitched(c["T"], C, torch.uint8)
                q.copy_((torch.randn(c["T"], C, generator=g, device="cuda") * 60).clamp(-448, 448)
                        .to(torch.float8_e4m3fn).view(torch.uint8))
                s["q"] = q
                s["s"] = torch.rand(-(-C // 128), c["T"], generator=g, device="cuda") * 0.02 + 0.002
            return s
        s["rows"] = _randn(g, P, C, _dt(c["rows"]))
        s["rows"][int(offsets[-1]):] = float("nan")  # rows that no expert owns are never written
        if kind == "combine_grad" or c["weighted"]:
            s["w"] = w
        if kind == "combine_grad":
            s["dy"] = _randn(g, c["T"], C, _dt(c["out"]), 1e-3)
        return s
    if kind == "clip":
        sizes = _sizes(c)
        kinds = [{"bf16": torch.bfloat16, "f32": torch.float32}.get(c["types"]) or
                 (torch.bfloat16 if i % 2 else torch.float32) for i in range(len(sizes))]
        s["grads"] = [(torch.randn(n, generator=g, device="cuda") * 1e-3).to(t) for n, t in zip(sizes, kinds)]
        # the clipped gradients go into one flat buffer, where the optimizer takes them from
        s["flat"] = torch.zeros(c["total"], dtype=_dt(c["out"]), device="cuda")
        s["outs"] = list(torch.split(s["flat"], sizes))
        s["max_norm"] = (0.5 if c["clips"] else 2.0) * 1e-3 * math.sqrt(c["total"])
        s["plan"] = {}  # what a program keeps between steps: the package's table of these tensors
        return s
    M, C = c["M"], c["C"]
    p = _dt(c["param"])
    res = _dt(c["res"])
    s["x"] = _randn(g, M, C, res)
    if c["pre"]:
        s["w_pre"] = (1 + 0.1 * torch.randn(C, generator=g, device="cuda")).to(p)
    if c["post"] != "none":
        s["f"] = _randn(g, M, C, torch.bfloat16)
    if c["post"] == "norm":
        s["w_post"] = (1 + 0.1 * torch.randn(C, generator=g, device="cuda")).to(p)
    if c["gate"] == "channel":
        s["gate"] = (0.5 + 0.2 * torch.randn(C, generator=g, device="cuda")).to(p)
    elif c["gate"] == "row":
        s["gate"] = _randn(g, M, C, torch.bfloat16, 0.5)
    if kind == "norm_grad":  # x is the residual stream after the sum; the statistics are those of the forward
        s["rstd_pre"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS_NORM) if c["pre"] else None
        s["rstd_post"] = torch.rsqrt(s["f"].float().square().mean(1) + EPS_NORM) if c["post"] == "norm" else None
        s["dn"] = _randn(g, M, C, torch.bfloat16, 1e-3) if c["pre"] else None
        s["dx_out"] = _randn(g, M, C, res, 1e-3)
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _plain_sort(ids, E):
    ids = ids.reshape(-1)
    kept = (ids >= 0) & (ids < E)
    key = torch.where(kept, ids.long(), torch.full_like(ids, E).long())
    order = torch.argsort(key, stable=True)  # dropped pairs come last
    counts = (key[:, None] == torch.arange(E, device=key.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    rank = torch.empty_like(order)
    rank[order] = torch.arange(order.numel(), device=order.device)
    row_of = torch.where(kept, rank, -1 - rank)
    slot_of = torch.where(kept[order], order, -1 - order)
    return offsets.to(torch.int32), row_of.to(torch.int32), slot_of.to(torch.int32)


def _any_row(row_of):
    """The row of every pair, also of the dropped ones."""
    r = row_of.long()
    return torch.where(r < 0, -1 - r, r)


def _plain_combine(s, c):
    r = s["row_of"].view(c["T"], c["K"])
    v = s["rows"][_any_row(r)].float()
    v = torch.where((r < 0)[..., None], torch.zeros_like(v), v)
    if c["weighted"]:
        v = v * s["w"][..., None]
    return v.sum(1).to(_dt(c["out"]))


def _plain_combine_grad(s, c):
    r = s["row_of"].view(c["T"], c["K"])
    dropped = (r < 0)[..., None]
    at = _any_row(r)
    dy = s["dy"].float()[:, None, :]
    v = s["rows"][at].float()
    v = torch.where(dropped, torch.zeros_like(v), v)
    dw = (v * dy).sum(-1)
    dr = torch.where(dropped, torch.zeros_like(v), s["w"][..., None] * dy)
    out = torch.empty(c["T"] * c["K"], c["C"], dtype=_dt(c["rows"]), device=dr.device)
    out[at.reshape(-1)] = dr.reshape(-1, c["C"]).to(out.dtype)
    return {"drows": out, "dweights": dw}


def _plain_quantize(n, pow2):
    M, C = n.shape
    G = -(-C // 128)
    t = torch.nn.functional.pad(n, (0, G * 128 - C)).view(M, G, 128)
    s = t.abs().amax(2) / E4M3_MAX
    if pow2:
        m, e = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    s = torch.where(t.abs().amax(2) == 0, torch.ones_like(s), s)
    q = (t / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view(M, G * 128)[:, :C]
    return q.to(torch.float8_e4m3fn), s.t().contiguous()


def _plain_norm(s, c):
    x = s["x"].float()
    out = {}
    if c["post"] != "none":
        u = s["f"].float()
        if c["post"] == "norm":
            r = torch.rsqrt(u.square().mean(1) + EPS_NORM)
            out["rstd_post"] = r
            u = u * r[:, None] * s["w_post"].float()
        if c["gate"] != "none":
            u = u * s["gate"].float()
        x = x + ALPHA * u
        out["x"] = x.to(_dt(c["res"]))
    if c["pre"]:
        r = torch.rsqrt(x.square().mean(1) + EPS_NORM)
        out["rstd_pre"] = r
        n = x * r[:, None] * s["w_pre"].float()
        out["n"] = n.to(torch.bfloat16)
        if c["quant"] != "none":
            out["q"], out["s"] = _plain_quantize(n, c["quant"] == "pow2")
    return out


def _plain_norm_grad(s, c):
    out = {}
    g = s["dx_out"].float()
    if c["pre"]:
        dn, xh = s["dn"].float(), s["x"].float() * s["rstd_pre"][:, None]
        out["dw_pre"] = (dn * xh).sum(0)
        v = dn * s["w_pre"].float()
        g = g + s["rstd_pre"][:, None] * (v - xh * (v * xh).mean(1, keepdim=True))
    out["dx"] = g.to(_dt(c["res"]))
    if c["post"] == "none":
        return out
    d = ALPHA * g
    f = s["f"].float()
    u = f
    if c["post"] == "norm":
        fh = f * s["rstd_post"][:, None]
        u = fh * s["w_post"].float()
    if c["gate"] == "channel":
        out["dgate"] = (d * u).sum(0)
    elif c["gate"] == "row":
        out["dgate"] = (d * u).to(torch.bfloat16)
    if c["gate"] != "none":
        d = d * s["gate"].float()
    if c["post"] == "norm":
        out["dw_post"] = (d * fh).sum(0)
        v = d * s["w_post"].float()
        d = s["rstd_post"][:, None] * (v - fh * (v * fh).mean(1, keepdim=True))
    out["df"] = d.to(torch.bfloat16)
    return out


def _plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "sort":
        o, r, t = _plain_sort(s["ids"], c["E"])
        return {"offsets": o, "row_of": r.view(c["T"], c["K"]), "slot_of": t}
    if kind == "dispatch":
        t = s["slot_of"].long()
        dropped = t < 0
        tok = torch.where(dropped, -1 - t, t) // c["K"]
        if c["type"] == "bf16":
            v = s["x"][tok]
            return torch.where(dropped[:, None], torch.zeros_like(v), v)
        v = s["q"][tok]
        v = torch.where(dropped[:, None], torch.zeros_like(v), v)
        sc = s["s"][:, tok]
        return {"q": v.view(torch.float8_e4m3fn), "s": torch.where(dropped[None, :], torch.ones_like(sc), sc)}
    if kind == "combine":
        return _plain_combine(s, c)
    if kind == "combine_grad":
        return _plain_combine_grad(s, c)
    if kind == "clip":
        norm = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt()
        coef = (s["max_norm"] / (norm + EPS_CLIP)).clamp(max=1.0)
        [o.copy_(t.float() * coef) for o, t in zip(s["outs"], s["grads"])]
        return {"norm": norm, "grads": s["flat"]}
    return _plain_norm(s, c) if kind == "norm" else _plain_norm_grad(s, c)


# --------------------------------------------------------------------------
# the package's calls
# --------------------------------------------------------------------------
def _called(s):
    import fp8_fine_grained_quantize_amd as fb

    c = s["case"]
    kind = c["kind"]
    if kind == "sort":
        offsets, row_of, slot_of = fb.moe_sort(s["ids"], c["E"])
        return {"offsets": offsets, "row_of": row_of, "slot_of": slot_of}
    if kind in ("dispatch", "combine", "combine_grad"):
        row_of = s["row_of"].view(c["T"], c["K"])
    if kind == "dispatch":
        if c["type"] == "bf16":
            return fb.moe_dispatch(s["x"], row_of)
        q, sc = fb.moe_dispatch_fp8(s["q"], s["s"], row_of, s["slot_of"])
        return {"q": q.view(torch.float8_e4m3fn), "s": sc}
    if kind == "combine":
        return fb.moe_combine(s["rows"], row_of, s["w"] if c["weighted"] else None, out_dtype=_dt(c["out"]))
    if kind == "combine_grad":
        dr, dw = fb.moe_combine_backward(s["dy"], s["rows"], row_of, s["w"])
        return {"drows": dr, "dweights": dw}
    if kind == "clip":
        if "table" not in s["plan"]:
            s["plan"]["table"] = fb.grad_table(s["grads"], outs=s["outs"])
        return {"norm": fb.clip_grad_norm(s["plan"]["table"], s["max_norm"], eps=EPS_CLIP), "grads": s["flat"]}
    if kind == "norm":
        r = fb.residual_norm(s["x"], w_pre=s.get("w_pre"), f=s.get("f"), w_post=s.get("w_post"), gate=s.get("gate"),
                             alpha=ALPHA, eps=EPS_NORM, quantize=c["quant"] != "none", pow2=c["quant"] == "pow2")
        out = {"rstd_post": r.rstd_post, "rstd_pre": r.rstd_pre, "n": r.n, "s": r.s,
               "x": r.x if c["post"] != "none" else None,
               "q": None if r.q is None else r.q.view(torch.float8_e4m3fn)}
    else:
        r = fb.residual_norm_backward(s["x"], dx_out=s["dx_out"], dn=s["dn"], rstd_pre=s["rstd_pre"],
                                      w_pre=s.get("w_pre"), f=s.get("f"), rstd_post=s["rstd_post"],
                                      w_post=s.get("w_post"), gate=s.get("gate"), alpha=ALPHA)
        out = {"dx": r.dx, "df": r.df, "dw_pre": r.dw_pre, "dw_post": r.dw_post, "dgate": r.dgate}
    return {k: v for k, v in out.items() if v is not None}


def run(state):
    return _called(state) if own else _plain(state)


# --------------------------------------------------------------------------
# what a pass cannot do without, each input read once, each output written once
# --------------------------------------------------------------------------
def work(case):
    c = case
    kind = c["kind"]
    if kind == "sort":
        P = c["T"] * c["K"]
        return {"bytes": P * ((4 if c["ids"] == "int32" else 8) + 8) + 4 * (c["E"] + 1), "flops": P}
    if kind in ("dispatch", "combine", "combine_grad"):
        T, K, C = c["T"], c["K"], c["C"]
        P = T * K
        if kind == "dispatch":
            if c["type"] == "bf16":
                return {"bytes": 2 * C * (T + P) + 4 * P, "flops": 0}
            return {"bytes": (C + 4 * (-(-C // 128))) * (T + P) + 8 * P, "flops": 0}
        rb, ob = (2 if c["rows"] == "bf16" else 4), (2 if c["out"] == "bf16" else 4)
        if kind == "combine":
            return {"bytes": P * C * rb + T * C * ob + P * (8 if c["weighted"] else 4), "flops": 2 * P * C}
        return {"bytes": 2 * P * C * rb + T * C * ob + 12 * P, "flops": 3 * P * C}
    if kind == "clip":
        at = {"bf16": 2.0, "f32": 4.0}
        if c["types"] == "mixed":
            got = sum(n * (2 if i % 2 else 4) for i, n in enumerate(_sizes(c)))
        else:
            got = c["total"] * at[c["types"]]
        # the norm needs every value before the first one can be scaled: two reads
        return {"bytes": 2 * got + c["total"] * at[c["out"]], "flops": 3 * c["total"]}
    n = c["M"] * c["C"]
    rb = 2 if c["res"] == "bf16" else 4
    if kind == "norm":
        b = n * rb + (n * (2 + rb) if c["post"] != "none" else 0) + (2 * n if c["gate"] == "row" else 0)
        if c["pre"]:
            b += 2 * n + (n + 4 * c["M"] * (-(-c["C"] // 128)) if c["quant"] != "none" else 0)
        return {"bytes": b, "flops": 10 * n}
    b = 2 * n * rb + (n * (2 + rb) if c["pre"] else 0) + (4 * n if c["post"] != "none" else 0)
    return {"bytes": b + (4 * n if c["gate"] == "row" else 0), "flops": 20 * n}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    c = case
    kind = c["kind"]
    if kind == "sort":
        return None  # whole numbers
    s = prepare(case, seed)
    with torch.no_grad():
        if kind == "dispatch":
            return _exact_dispatch(s, c)
        if kind in ("combine", "combine_grad"):
            return _exact_moe(s, c)
        if kind == "clip":
            total = sum(float((t.double() ** 2).sum()) for t in s["grads"])
            norm = math.sqrt(total)
            coef = min(1.0, s["max_norm"] / (norm + EPS_CLIP))
            return {"norm": norm, "grads": torch.cat([t.double() * coef for t in s["grads"]])}
        return _exact_norm(s, c) if kind == "norm" else _exact_norm_grad(s, c)


def _exact_dispatch(s, c):
    """One slot of all tokens at a time; rows that no expert owns are zero."""
    T, K, C = c["T"], c["K"], c["C"]
    row = s["row_of"].view(T, K).long()
    x = s["x"].double() if c["type"] == "bf16" else s["q"].view(torch.float8_e4m3fn).double()
    out = torch.zeros(T * K, C, dtype=torch.float64, device="cuda")
    sc = torch.ones(-(-C // 128), T * K, dtype=torch.float64, device="cuda")
    for k in range(K):
        t = torch.nonzero(row[:, k] >= 0).squeeze(1)
        out[row[t, k]] = x[t]
        if c["type"] == "fp8":
            sc[:, row[t, k]] = s["s"][:, t].double()
    return out if c["type"] == "bf16" else {"q": out, "s": sc}


def _exact_moe(s, c):
    """One slot of all tokens at a time."""
    T, K, C = c["T"], c["K"], c["C"]
    row = s["row_of"].view(T, K).long()
    grad = c["kind"] == "combine_grad"
    if grad:
        dy = s["dy"].double()
        dr = torch.zeros(T * K, C, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    else:
        y = torch.zeros(T, C, dtype=torch.float64, device="cuda")
    for k in range(K):
        t = torch.nonzero(row[:, k] >= 0).squeeze(1)
        r = row[t, k]
        v = s["rows"][r].double()
        if grad:
            dw[t, k] = (v * dy[t]).sum(1)
            dr[r] = dy[t] * s["w"][t, k].double()[:, None]
        else:
            y[t] += v * s["w"][t, k].double()[:, None] if c["weighted"] else v
    return {"drows": dr, "dweights": dw} if grad else y


def _exact_norm(s, c):
    out = {}
    z = s["x"].double()
    C = c["C"]
    if c["post"] != "none":
        f = s["f"].double()
        if c["post"] == "norm":
            out["rstd_post"] = 1.0 / torch.sqrt((f * f).sum(1) / C + EPS_NORM)
            f = torch.einsum("mc,m,c->mc", f, out["rstd_post"], s["w_post"].double())
        if "gate" in s:
            f = f * s["gate"].double()
        z = z + ALPHA * f
        out["x"] = z
    if c["pre"]:
        out["rstd_pre"] = 1.0 / torch.sqrt((z * z).sum(1) / C + EPS_NORM)
        n = torch.einsum("mc,m,c->mc", z, out["rstd_pre"], s["w_pre"].double())
        out["n"] = n
        if c["quant"] != "none":
            sc, q = [], torch.empty_like(n)
            for a in range(0, C, 128):
                m = n[:, a:a + 128].abs().max(1).values
                v = torch.exp2(torch.ceil(torch.log2(m / E4M3_MAX))) if c["quant"] == "pow2" else m / E4M3_MAX
                v = torch.where(m == 0, torch.ones_like(v), v)
                sc.append(v)
                q[:, a:a + 128] = n[:, a:a + 128] / v[:, None]  # before it is rounded to a code
            out["q"], out["s"] = q, torch.stack(sc)
    return out


def _exact_norm_grad(s, c):
    """From n_j = z_j r w_j with r = (mean(z^2) + eps)^-1/2: dr/dz_i = -r^3 z_i / C."""
    out = {}
    C = c["C"]
    total = s["dx_out"].double()
    if c["pre"]:
        z, r, w, dn = s["x"].double(), s["rstd_pre"].double()[:, None], s["w_pre"].double(), s["dn"].double()
        out["dw_pre"] = (dn * z * r).sum(0)
        total = total + dn * w * r - z * r ** 3 / C * (dn * w * z).sum(1, keepdim=True)
    out["dx"] = total
    if c["post"] == "none":
        return out
    f = s["f"].double()
    gate = s["gate"].double() if "gate" in s else torch.ones((), dtype=torch.float64, device="cuda")
    if c["post"] == "norm":
        r, w = s["rstd_post"].double()[:, None], s["w_post"].double()
        du = total * gate * ALPHA
        out["dw_post"] = (du * f * r).sum(0)
        out["df"] = du * w * r - f * r ** 3 / C * (du * w * f).sum(1, keepdim=True)
        dgate = total * ALPHA * f * r * w
    else:
        out["df"] = total * gate * ALPHA
        dgate = total * ALPHA * f
    if c["gate"] == "channel":
        out["dgate"] = dgate.sum(0)
    elif c["gate"] == "row":
        out["dgate"] = dgate
    return out
