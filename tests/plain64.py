"""The 8-bit operators and the norms around a block in numpy float64, each with the
error bound its fp32 kernel has to keep, element by element.

Bounds. u = 2^-24 is half a step of fp32 relative to the value; a sum of n terms taken in
any order by at most k dependent additions is off by at most k u sum|terms|. A thread of
the kernels adds at most 80 values of its own and the partial sums of a row join in at most
14 more steps, so k <= 94 and K_SUM = 100 covers the product or square inside each term
too. rsqrtf and the fast exponential and divide of SiLU add a few fp32 steps each.
"""
import numpy as np

U = 2.0 ** -24
K_SUM = 100
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def codes(v):
    """Rows v (..., K) -> (codes, scale): scale = max|v| / 127, code = rint(127 v / max|v|)."""
    v = np.asarray(v, dtype=np.float64)
    bad = ~np.isfinite(v).all(-1)
    amax = np.abs(np.where(bad[..., None], 0.0, v)).max(-1)
    q = np.rint(127.0 * np.where(bad[..., None], 0.0, v) / np.where(amax == 0, 1.0, amax)[..., None])
    return q, np.where(bad, np.nan, amax / 127.0)


def check_codes(q, scale, ref, tol):
    """q, scale: the kernel's codes of rows whose exact values are ref, each known to within
    tol. The kernel quantises its own values v, |v - ref| <= tol: |scale - amax/127| is at most
    max(tol)/127 and one rounding, and |q scale - v| at most half a scale, the codes' step (and
    the roundings of mul and scale, 4 u of a value of at most 127 scale)."""
    q, scale = np.asarray(q, dtype=np.float64), np.asarray(scale, dtype=np.float64)
    assert np.abs(q).max(initial=0) <= 127
    amax = np.abs(ref).max(-1)
    assert (np.abs(scale - amax / 127) <= (tol.max(-1) * (1 + U) + 2 * U * amax) / 127 + 2.0 ** -149).all()
    off = np.abs(q * scale[..., None] - ref)
    limit = 0.5 * scale[..., None] * (1 + 1e-6) + tol + 127 * 4 * U * scale[..., None] + 2.0 ** -140
    assert (off <= limit).all(), float((off - limit).max())


def linear(xq, xs, wq, ws, bias=None, addend=None):
    """-> (value, bound of the fp32 epilogue before the output's rounding)."""
    acc = np.asarray(xq, dtype=np.float64) @ np.asarray(wq, dtype=np.float64).T
    p = acc * np.asarray(xs, np.float64)[:, None] * np.asarray(ws, np.float64)[None, :]
    mag = np.abs(p)
    for more in (bias, addend):
        if more is not None:
            p = p + np.asarray(more, np.float64)
            mag = mag + np.abs(np.asarray(more, np.float64))
    return p, 6 * U * mag  # int -> float, two scales, two sums; one more for their products


def norm(v, kind, eps, dv=0.0):
    """N(v) over the last axis -> (value, bound), dv bounding the error v already has."""
    n = v.shape[-1]
    mu, dmu = 0.0, 0.0
    if kind == "none":
        return v, np.broadcast_to(np.asarray(dv), v.shape)
    dv = np.broadcast_to(np.asarray(dv, dtype=np.float64), v.shape)
    if kind == "layer":
        mu = v.sum(-1, keepdims=True) / n
        dmu = K_SUM * U * np.abs(v).sum(-1, keepdims=True) / n + dv.mean(-1, keepdims=True)
    d = v - mu
    dd = dv + dmu + U * np.abs(d)
    ms = (d * d).sum(-1, keepdims=True) / n + eps
    # relative error of the mean square (2 |d| dd per term and the sum's own), halved by the root
    rel = ((2 * np.abs(d) * dd + dd * dd).sum(-1, keepdims=True) / n / ms + K_SUM * U) / 2 + 4 * U
    out = d / np.sqrt(ms)
    return out, dd / np.sqrt(ms) + np.abs(out) * (rel + 2 * U)


def block_norm(x, y=None, w_post=None, gate=None, alpha=1.0, post="rms", w_pre=None, scale=None, shift=None,
               pre="rms", eps=1e-6):
    """x, y: (batch, n, C); gate, scale, shift: (batch, C). -> ((r, dr) or None, (h, dh))."""
    f = lambda t: None if t is None else np.asarray(t, dtype=np.float64)  # noqa: E731
    x, y, w_post, gate, w_pre, scale, shift = map(f, (x, y, w_post, gate, w_pre, scale, shift))
    r, dr, first = x, np.zeros_like(x), None
    if y is not None:
        N, dN = norm(y, post, eps)
        g = (1.0 if gate is None else gate[:, None, :]) * (1.0 if w_post is None else w_post)
        r = alpha * x + g * N
        dr = np.abs(g) * dN + 4 * U * (np.abs(alpha * x) + np.abs(g * N))
        first = (r, dr)
    N, dN = norm(r, pre, eps, dr)
    a = (1.0 if w_pre is None else w_pre) * (1.0 if scale is None else 1.0 + scale[:, None, :])
    s = 0.0 if shift is None else shift[:, None, :]
    h = N * a + s
    # a = w (1 + scale) is off by u of its summands each
    da = 2 * U * ((np.abs(w_pre) if w_pre is not None else 1.0) * (1 + (0 if scale is None else np.abs(scale[:, None, :]))))
    return first, (h, np.abs(a) * dN + np.abs(N) * da + 3 * U * (np.abs(N * a) + np.abs(s)))


def gate_norm(y, z, w, group, eps):
    """-> (value, bound). SiLU by the fast exponential and divide: __expf is within
    2 + floor(1.173 |z|) fp32 steps, the divide within 2."""
    y, z, w = (np.asarray(t, dtype=np.float64) for t in (y, z, w))
    v = y * z / (1 + np.exp(-z))
    dv = np.abs(v) * 2 * U * (8 + 1.2 * np.abs(z))
    M, C = v.shape
    N, dN = norm(v.reshape(M, C // group, group), "rms", eps, dv.reshape(M, C // group, group))
    N, dN = N.reshape(M, C), dN.reshape(M, C)
    return N * w, np.abs(w) * dN + 3 * U * np.abs(N * w)
