"""Plain 64-bit forms of the operators around the GEMMs (NumPy, CPU), and the
rounding-error bounds that the GPU tests hold their outputs to.

U is the unit roundoff of FP32, UB that of BF16.  A sum of m products formed
in any order by FMAs and additions differs from the exact one by at most
m U * sum |products| (to first order, which a factor of 2 more than covers at
these sizes); each further FP32 operation adds one U of its result's
magnitude, and a final rounding to BF16 one UB.
"""
import numpy as np

U, UB = 2.0 ** -24, 2.0 ** -8  # significands of 24 and 8 bits


def sort_pairs(ids, E):
    """(offsets, row_of [T][K], slot_of) by walking the pairs one by one."""
    T, K = ids.shape
    flat = ids.reshape(-1)
    kept = [p for p in range(T * K) if 0 <= flat[p] < E]
    dropped = [p for p in range(T * K) if not 0 <= flat[p] < E]
    by_expert = sorted(kept, key=lambda p: flat[p])  # Python's sort is stable
    offsets = np.zeros(E + 1, dtype=np.int64)
    for p in kept:
        offsets[flat[p] + 1] += 1
    offsets = np.cumsum(offsets)
    row_of = np.zeros(T * K, dtype=np.int64)
    slot_of = np.zeros(T * K, dtype=np.int64)
    for r, p in enumerate(by_expert):
        row_of[p], slot_of[r] = r, p
    for i, p in enumerate(dropped):
        r = len(kept) + i
        row_of[p], slot_of[r] = -1 - r, -1 - p
    return offsets, row_of.reshape(T, K), slot_of


def combine(rows, row_of, w):
    """(y, sum of magnitudes) in 64 bits; w None: all one."""
    T, K = row_of.shape
    y = np.zeros((T, rows.shape[1]))
    mag = np.zeros_like(y)
    for t in range(T):
        for k in range(K):
            if row_of[t, k] >= 0:
                v = rows[row_of[t, k]].astype(np.float64) * (1.0 if w is None else float(w[t, k]))
                y[t] += v
                mag[t] += np.abs(v)
    return y, mag


def combine_backward(dy, rows, row_of, w):
    """(drows, dw, sum of magnitudes of dw's terms) in 64 bits."""
    T, K = row_of.shape
    dr = np.zeros(rows.shape)
    dw = np.zeros((T, K))
    mag = np.zeros((T, K))
    for t in range(T):
        for k in range(K):
            r = row_of[t, k]
            if r >= 0:
                dr[r] = float(w[t, k]) * dy[t].astype(np.float64)
                terms = dy[t].astype(np.float64) * rows[r].astype(np.float64)
                dw[t, k], mag[t, k] = terms.sum(), np.abs(terms).sum()
    return dr, dw, mag


def norm_forward(x, w_pre=None, f=None, w_post=None, gate=None, alpha=1.0, eps=1e-6):
    """dict of x, n, rstd_post, rstd_pre (64 bits) and `mag`, |x| + |alpha gate u|."""
    x = x.astype(np.float64)
    out = {"rstd_post": None, "rstd_pre": None, "n": None, "mag": np.abs(x)}
    if f is not None:
        u = f.astype(np.float64)
        if w_post is not None:
            r = 1.0 / np.sqrt(np.mean(u * u, axis=1) + eps)
            out["rstd_post"] = r
            u = u * r[:, None] * w_post.astype(np.float64)
        if gate is not None:
            u = u * gate.astype(np.float64)
        out["mag"] = np.abs(x) + np.abs(alpha * u)
        x = x + alpha * u
    out["x"] = x
    if w_pre is not None:
        r = 1.0 / np.sqrt(np.mean(x * x, axis=1) + eps)
        out["rstd_pre"] = r
        out["n"] = x * r[:, None] * w_pre.astype(np.float64)
    return out


def _rms_backward(v, z, r):
    """Gradient into z of z r w for the gradient v = dn w, with r(z)."""
    h = z * r[:, None]
    return r[:, None] * (v - h * np.mean(v * h, axis=1, keepdims=True))


def norm_backward(x, dx_out=None, dn=None, rstd_pre=None, w_pre=None, f=None, rstd_post=None, w_post=None, gate=None,
                  alpha=1.0):
    """dict of the gradients in 64 bits, from the statistics as given."""
    g64 = lambda t: None if t is None else t.astype(np.float64)  # noqa: E731
    x, dx_out, dn, rstd_pre, w_pre, f, rstd_post, w_post, gate = map(
        g64, (x, dx_out, dn, rstd_pre, w_pre, f, rstd_post, w_post, gate))
    g = np.zeros_like(x) if dx_out is None else dx_out.copy()
    out = dict.fromkeys(("df", "dw_pre", "dw_post", "dgate"))
    if w_pre is not None:
        out["dw_pre"] = (dn * x * rstd_pre[:, None]).sum(0)
        g = g + _rms_backward(dn * w_pre, x, rstd_pre)
    out["dx"] = g
    if f is not None:
        d = alpha * g
        u = f
        if w_post is not None:
            u = f * rstd_post[:, None] * w_post
        if gate is not None:
            out["dgate"] = d * u if gate.ndim == 2 else (d * u).sum(0)
            d = d * gate
        if w_post is not None:
            out["dw_post"] = (d * f * rstd_post[:, None]).sum(0)
            d = _rms_backward(d * w_post, f, rstd_post)
        out["df"] = d
    return out
