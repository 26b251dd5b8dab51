"""FP64 oracle of the block norms: h' = alpha h + gate * N_post(b),
n = N_pre(h') (1 + scale) + shift, and their gradients."""

import numpy as np


def normalise(v, kind, eps):
    """(N(v), 1 / deviation per row) for kind None, 'rms' or 'layer'."""
    v = np.asarray(v, dtype=np.float64)
    if kind is None:
        return v, np.ones((v.shape[0], 1))
    if kind == "layer":
        v = v - v.mean(1, keepdims=True)
    r = 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    return v * r, r


def normalise_backward(g, v, kind, eps):
    """Gradient at v of sum(g * N(v))."""
    u, r = normalise(v, kind, eps)
    if kind is None:
        return np.asarray(g, dtype=np.float64)
    d = g - u * (g * u).mean(1, keepdims=True)
    if kind == "layer":
        d = d - g.mean(1, keepdims=True)
    return r * d


def rows_of(mod, M, seg, other):
    """The modulation row of each of M rows ([S, D] -> [M, D])."""
    return other if mod is None else np.asarray(mod, dtype=np.float64)[np.arange(M) // seg]


def residual(h, b, gate, alpha, eps, post, seg):
    M = h.shape[0]
    return alpha * np.asarray(h, np.float64) + rows_of(gate, M, seg, 1.0) * normalise(b, post, eps)[0]


def modulated(h, scale, shift, eps, pre, seg):
    M = h.shape[0]
    return normalise(h, pre, eps)[0] * (1.0 + rows_of(scale, M, seg, 0.0)) + rows_of(shift, M, seg, 0.0)


def segment_sums(v, seg):
    return np.add.reduceat(v, np.arange(0, v.shape[0], seg), axis=0)


def backward(dn, dh_out, h_out, b, gate, scale, alpha, eps, post, pre, seg):
    """(dh, db, dgate, dscale, dshift) in FP64; None where there is none."""
    M = h_out.shape[0]
    dh = np.zeros(h_out.shape) if dh_out is None else np.asarray(dh_out, np.float64)
    dscale = dshift = db = dgate = None
    if pre is not None:
        dn = np.asarray(dn, np.float64)
        dh = dh + normalise_backward(dn * (1.0 + rows_of(scale, M, seg, 0.0)), h_out, pre, eps)
        dscale = segment_sums(dn * normalise(h_out, pre, eps)[0], seg)
        dshift = segment_sums(dn, seg)
    if b is not None:
        dgate = segment_sums(dh * normalise(b, post, eps)[0], seg)
        db = normalise_backward(rows_of(gate, M, seg, 1.0) * dh, b, post, eps)
    return alpha * dh, db, dgate, dscale, dshift
