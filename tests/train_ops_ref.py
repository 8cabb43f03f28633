"""Plain fp64 forms of the operators around a layer in a training step, and
bounds on a device result's distance from them, counted in roundings.

u = 2^-24 is the largest relative error of one fp32 rounding, HALF[t] that of a
rounding to t.  A sum of n terms by any fixed tree of depth d is off by at most
d u times the sum of the terms' magnitudes (first order; the small factors
below leave room for the second).
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
# Depth of a row sum: 16 columns a thread, 5 shuffles, 16 warps, and the
# product's rounding.
ROW = 16 + 5 + 16 + 1
# r = 1 / rms: half of the row sum's relative error (the root), the 1/D and
# eps roundings (2), and rsqrtf's 2 ulp (4 u).
RMS = ROW / 2 + 2 + 4


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def embed_backward(ids, dout, dE, scale, V):
    """(dE + scale sum dout, the bound): c additions for c tokens of an id, one
    product, one addition to dE."""
    out, mag, cnt = dE.copy(), np.abs(dE), np.zeros(V)
    ok = (ids >= 0) & (ids < V)
    np.add.at(out, ids[ok], scale * dout[ok])
    np.add.at(mag, ids[ok], abs(scale) * np.abs(dout[ok]))
    np.add.at(cnt, ids[ok], 1)
    return out, np.where(cnt[:, None] > 0, (cnt[:, None] + 4) * U * mag, 0.0)


def norm_forward(x, f, w_post, gate, res_scale, w_pre, eps):
    """x', h and their bounds before the rounding to their types."""
    T, D = x.shape
    y = np.zeros_like(x)
    if f is not None:
        y = f if w_post is None else f / np.sqrt((f * f).mean(1, keepdims=True) + eps) * w_post
    g = np.ones(T) if gate is None else gate
    xo = res_scale * x + g[:, None] * y
    mag = np.abs(res_scale * x) + np.abs(g[:, None] * y)
    bx = (RMS + 5) * U * mag          # r, two products of y, product and sum of x'
    if w_pre is None:
        return xo, None, bx, None
    r = 1.0 / np.sqrt((xo * xo).mean(1, keepdims=True) + eps)
    h = xo * r * w_pre
    # the root of the sum of squares moves by at most |bx| in the 2-norm
    norm = np.sqrt((xo * xo).sum(1, keepdims=True) + D * eps)
    rel_r = RMS * U + np.linalg.norm(bx, axis=1, keepdims=True) / norm
    return xo, h, bx, np.abs(w_pre * r) * bx + np.abs(h) * (rel_r + 4 * U)


def norm_backward(xo, f, w_post, gate, res_scale, w_pre, eps, dx_out, dh):
    """{name: (value, bound)} of dx, df, dgate, dw_pre, dw_post (the sums over
    the tokens, without what they are added to)."""
    T, D = (xo if xo is not None else dx_out).shape
    G = np.zeros((T, D)) if dx_out is None else dx_out
    MG = np.abs(G)
    out = {}
    # tokens: at most T / 100 + 80 additions of one thread, its CTA and the join
    deep = T / 100 + 80
    if dh is not None:
        r = 1.0 / np.sqrt((xo * xo).mean(1, keepdims=True) + eps)
        a, xh = dh * w_pre, xo * r
        G = G + r * (a - xh * (a * xh).mean(1, keepdims=True))
        # c = r^2 sum(a x')/n: the sum's depth, a's rounding, r twice
        A = np.abs(a * xo).mean(1, keepdims=True)
        MG = MG + r * (np.abs(a) + r * r * A * np.abs(xo))
        out["dw_pre"] = ((dh * xh).sum(0), (deep + RMS + 3) * U * np.abs(dh * xh).sum(0))
    bG = (ROW + 3 * RMS + 8) * U      # relative to MG
    out["dx"] = (res_scale * G, (bG + 2 * U) * abs(res_scale) * MG)
    g = np.ones((T, 1)) if gate is None else gate[:, None]
    if f is None:
        out["df"] = (g * G, (bG + 2 * U) * np.abs(g) * MG)
        return out
    w = np.ones(D) if w_post is None else w_post
    rf = np.ones((T, 1)) if w_post is None else 1.0 / np.sqrt((f * f).mean(1, keepdims=True) + eps)
    fh = f * rf
    q = (G * w * fh).sum(1, keepdims=True)
    Q = (MG * np.abs(w * fh)).sum(1, keepdims=True)
    bq = bG + (ROW + RMS + 4) * U
    out["dgate"] = (q[:, 0], bq * Q[:, 0])
    if w_post is None:
        out["df"] = (g * G, (bG + 3 * U) * np.abs(g) * MG)
    else:
        out["df"] = (g * rf * (G * w - fh * q / D),
                     (bq + (2 * RMS + 8) * U) * np.abs(g) * rf * (MG * np.abs(w) + np.abs(fh) * Q / D))
        out["dw_post"] = ((g * G * fh).sum(0),
                          (bG + (deep + RMS + 4) * U) * (np.abs(g) * MG * np.abs(fh)).sum(0))
    return out


def adamw(p, g, m, v, lr, beta1, beta2, eps, step, weight_decay):
    """(p, m, v) after a step and their bounds."""
    mm, vv = np.abs(beta1 * m) + np.abs((1 - beta1) * g), beta2 * v + (1 - beta2) * g * g
    m, v = beta1 * m + (1 - beta1) * g, vv
    den = np.sqrt(v / (1 - beta2 ** step)) + eps
    upd = lr / (1 - beta1 ** step) * m / den
    # m: the constants, two products, a sum (and a gradient factor); v: three
    # products; den: half of v's, the root, its factor, the sum; the quotient
    # (2 ulp allowed), step size and two sums of p
    bm, bv = 5 * U * mm, 7 * U * vv
    bp = lr / (1 - beta1 ** step) * bm / den + np.abs(upd) * 16 * U + 4 * U * (np.abs(p) + np.abs(upd))
    return p - lr * weight_decay * p - upd, m, v, bp, bm, bv


def assert_within(got, ref, bound, name=""):
    """|got - ref| <= bound for every element (NaN in got fails)."""
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.size} beyond the bound, first at "
                           f"{tuple(np.argwhere(bad)[0])}: {got[bad][0]!r} for {ref[bad][0]!r} "
                           f"(bound {np.broadcast_to(bound, bad.shape)[bad][0]:.3e})")
