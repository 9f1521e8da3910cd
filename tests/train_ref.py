"""64-bit references of the fine-tuning operators (numpy float64 on the host,
written from their definitions; nothing here is shared with the library)."""
from __future__ import annotations

import numpy as np

MXINT8, MXFP8 = 0, 1
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def half_step(dtype_name):
    """Half a unit in the last place of a value, relative: bf16 2^-8, fp32 2^-24."""
    return {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[dtype_name]


def within(got, ref, bound, what):
    """Elementwise |got - ref| <= bound; NaN exactly where the reference has it."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    ok = ~np.isnan(ref)
    err = np.abs(got - ref)[ok]
    b = np.broadcast_to(np.asarray(bound, np.float64), ref.shape)[ok]
    bad = err > b
    if bad.any():
        i = int(np.argmax(err - b))
        raise AssertionError(f"{what}: {int(bad.sum())} of {err.size} outside; worst {err[i]:.3e} > {b[i]:.3e} "
                             f"(ref {ref[ok][i]:.6e})")


def bf16(v):
    """Round to nearest even to bf16, as float64."""
    b = np.asarray(v, np.float32).view(np.uint32).astype(np.uint64)
    nan = np.isnan(np.asarray(v, np.float32))
    r = ((b + 0x7fff + ((b >> 16) & 1)) & 0xffff0000).astype(np.uint32).view(np.float32).astype(np.float64)
    return np.where(nan, np.nan, r)


# ------------------------------------------------------------------ 8-bit checkpoints
def ckpt8(x, fmt):
    """(codes uint8, scale bytes, values float64) of x [.., K]."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1, keepdims=True)
    b = np.where(bad, 0.0, b)
    amax = np.abs(b).max(-1, keepdims=True)
    top = np.where(amax > 0, np.frexp(amax)[1] - 1, -127)
    X = np.maximum(top - (8 if fmt == MXFP8 else 0), -127).astype(np.int64)
    if fmt == MXINT8:
        q = np.clip(np.rint(np.ldexp(b, 6 - X)), -127, 127)
        codes = q.astype(np.int8).view(np.uint8)
        vals = np.ldexp(q, X - 6)
    else:
        v = np.ldexp(np.abs(b), -X)
        hi = np.minimum(np.searchsorted(E4M3, v), len(E4M3) - 1)
        lo = np.maximum(hi - 1, 0)
        dh, dl = E4M3[hi] - v, v - E4M3[lo]
        n = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
        codes = (n + np.where(np.signbit(b), 128, 0)).astype(np.uint8)
        vals = np.ldexp(E4M3[n], X) * np.where(np.signbit(b), -1.0, 1.0)
    scale = np.where(bad, 255, X + 127).astype(np.uint8)
    codes = np.where(bad, 0, codes).astype(np.uint8)
    vals = np.where(bad, np.nan, vals)
    return codes.reshape(x.shape), scale.reshape(*x.shape[:-1], -1), vals.reshape(x.shape)


# ------------------------------------------------------------------ gated activation
def _sigma(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def split(gu, inter):
    I = gu.shape[1] // 2
    return (gu[:, 0::2], gu[:, 1::2]) if inter else (gu[:, :I], gu[:, I:])


def join(a, b, inter):
    out = np.empty((a.shape[0], 2 * a.shape[1]))
    if inter:
        out[:, 0::2], out[:, 1::2] = a, b
    else:
        out[:, :a.shape[1]], out[:, a.shape[1]:] = a, b
    return out


def glu(gu, kind, alpha, limit, inter):
    g, u = split(np.asarray(gu, np.float64), inter)
    if kind == 0:
        return g * _sigma(g) * u
    g, u = np.where(g > limit, limit, g), np.clip(u, -limit, limit)
    return (u + 1) * g * _sigma(alpha * g)


def glu_grad(gu, dh, w, kind, alpha, limit, inter):
    """dgu, h, drow, and bounds of the fp32 evaluation error of dgu and h: with the
    exponent's argument rounded (|a g| 2^-24 relative each) and about one unit in
    the last place from each of exp2, the reciprocal and the products, sigma is
    within (|a g| + 8) 2^-23 of itself, and each result within that share of the
    sum of its terms' magnitudes."""
    g, u = split(np.asarray(gu, np.float64), inter)
    d = dh * w[:, None]
    al = alpha if kind == 1 else 1.0
    live_g = live_u = np.ones_like(g)
    if kind == 1:
        live_g, live_u = (~(g > limit)).astype(float), (~(np.abs(u) > limit)).astype(float)
        g, u = np.where(g > limit, limit, g), np.clip(u, -limit, limit) + 1
    s = _sigma(al * g)
    with np.errstate(invalid="ignore"):
        share = (np.abs(al * g) + 8) * 2.0 ** -23
        dg = live_g * d * u * s * (1 + al * g * (1 - s))
        du = live_u * d * g * s
        h = g * s * u
        # 1 - s is off by sigma's own absolute error
        eg = live_g * share * np.abs(d * u * s) * (1 + np.abs(al * g) * (1 - s) + np.abs(al * g) * s)
        eu = live_u * share * np.abs(d * g * s)
    return (join(dg, du, inter), h, (dh * h).sum(1)), (join(eg, eu, inter), share * np.abs(h))


# ------------------------------------------------------------------ block norms
def phi(gate, fn):
    return (gate, _sigma(gate), np.tanh(gate))[fn]


def slope(gate, fn):
    return (np.ones_like(gate), _sigma(gate) * (1 - _sigma(gate)), 1 - np.tanh(gate) ** 2)[fn]


def norm_forward(x, f, w_post, w_pre, gate, fn, alpha, eps, store):
    """store rounds the residual stream to its type."""
    rp = r = y = None
    if f is not None:
        z = f
        if w_post is not None:
            rp = 1 / np.sqrt((f ** 2).mean(1) + eps)
            z = f * rp[:, None] * w_post
        x = x + alpha * (1.0 if gate is None else phi(gate, fn)) * z
    if w_pre is not None:
        xs = store(x)
        r = 1 / np.sqrt((xs ** 2).mean(1) + eps)
        y = xs * r[:, None] * w_pre
    return x, y, rp, r


def norm_backward(dx_new, dy, x_new, f, rp, r, w_post, w_pre, gate, fn, alpha):
    """Gradients, and for each the sum of its terms' magnitudes (what fp32 errors scale with)."""
    out, mag = {}, {}
    H = x_new.shape[1]
    g = np.zeros_like(x_new) if dx_new is None else dx_new
    gm = np.abs(g)
    if w_pre is not None:
        n = x_new * r[:, None]
        out["dw_pre"], mag["dw_pre"] = (dy * n).sum(0), np.abs(dy * n).sum(0)
        a = dy * w_pre
        g = g + r[:, None] * (a - n * (a * n).sum(1, keepdims=True) / H)
        gm = gm + r[:, None] * (np.abs(a) + np.abs(n) * np.abs(a * n).sum(1, keepdims=True) / H)
    out["dx"], mag["dx"] = g, gm
    if f is None:
        return out, mag
    n = f if rp is None else f * rp[:, None]
    z = n if w_post is None else n * w_post
    p = np.ones((1, 1)) if gate is None else phi(gate, fn)
    if gate is not None:
        sl = slope(gate, fn)
        dg, dm = alpha * sl * g * z, abs(alpha) * np.abs(sl) * gm * np.abs(z)
        if gate.ndim == 1:
            dg, dm = dg.sum(0), dm.sum(0)
        elif gate.shape[1] == 1:
            dg, dm = dg.sum(1, keepdims=True), dm.sum(1, keepdims=True)
        out["dgate"], mag["dgate"] = dg, dm
    dz, dzm = alpha * p * g, np.abs(alpha * p) * gm
    if w_post is not None:
        out["dw_post"], mag["dw_post"] = (dz * n).sum(0), (dzm * np.abs(n)).sum(0)
        a, am = dz * w_post, dzm * np.abs(w_post)
        dz = rp[:, None] * (a - n * (a * n).sum(1, keepdims=True) / H)
        dzm = rp[:, None] * (am + np.abs(n) * (am * np.abs(n)).sum(1, keepdims=True) / H)
    out["df"], mag["df"] = dz, dzm
    return out, mag


# ------------------------------------------------------------------ adapters
def adapter_rows(ids, L):
    ids = np.asarray(ids)
    return {l: np.flatnonzero(ids == l) for l in np.unique(ids) if 0 <= l < L}


def adapter_forward(x, A, B, ids, scale, base, row_of):
    """out, t, and the sums of the magnitudes of their terms (base left out)."""
    R, (L, r, K), N = len(ids), A.shape, B.shape[1]
    xr = x if row_of is None else x[row_of]
    t, tm, d, dm = np.zeros((R, r)), np.zeros((R, r)), np.zeros((R, N)), np.zeros((R, N))
    for l, rows in adapter_rows(ids, L).items():
        t[rows], tm[rows] = xr[rows] @ A[l].T, np.abs(xr[rows]) @ np.abs(A[l]).T
        d[rows], dm[rows] = scale[l] * (t[rows] @ B[l].T), abs(scale[l]) * (tm[rows] @ np.abs(B[l]).T)
    return (d if base is None else base + d), t, dm, tm


def adapter_backward(dy, x, t, A, B, ids, scale, dx_base, row_of):
    """dx, dA, dB and the sums of the magnitudes of their terms (dx_base left out)."""
    R, (L, r, K), N = len(ids), A.shape, B.shape[1]
    xr = x if row_of is None else x[row_of]
    out = dict(dx=np.zeros((R, K)) if dx_base is None else dx_base.copy(), dA=np.zeros((L, r, K)), dB=np.zeros((L, N, r)))
    mag = dict(dx=np.zeros((R, K)), dA=np.zeros((L, r, K)), dB=np.zeros((L, N, r)))
    for l, rows in adapter_rows(ids, L).items():
        g, gm = dy[rows], np.abs(dy[rows])
        u, um = scale[l] * (g @ B[l]), abs(scale[l]) * (gm @ np.abs(B[l]))
        out["dx"][rows] += u @ A[l]
        mag["dx"][rows] = um @ np.abs(A[l])
        out["dA"][l], mag["dA"][l] = u.T @ xr[rows], um.T @ np.abs(xr[rows])
        out["dB"][l], mag["dB"][l] = scale[l] * (g.T @ t[rows]), abs(scale[l]) * (gm.T @ np.abs(t[rows]))
    return out, mag
