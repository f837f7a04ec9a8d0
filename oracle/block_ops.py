"""Float64 definitions of the operators around the delta-rule kernels, in numpy and
token by token: the gated linear recurrence with its gradients, the norms around a
block with theirs, and the delta rule on a cache of states.

Each comes with a bound on the rounding errors of a computation in 32 bits: the same
formula run over magnitudes, every product and sum adding its half step U = 2^-24
(``*_bound``).  The bounds assume nothing about the order of the sums but the counts named
beside them.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24            # half a step of fp32, relative
HALF_STEP = {"bfloat16": 2.0 ** -8, "float32": U}


def sequences(B: int, T: int, cu=None):
    """(row, state, first token, one past the last token) of every sequence."""
    if cu is None:
        return [(b, b, 0, T) for b in range(B)]
    return [(0, n, int(cu[n]), int(cu[n + 1])) for n in range(len(cu) - 1)]


# ---- gated linear recurrence ---------------------------------------------------

def scan(x, g, init=None, cu=None):
    """h_t = exp(g_t) h_{t-1} + x_t: (h [B, T, D], final [N, D], bound on h, bound on final).

    Bound: h_t is a sum of products of decays with an input.  Each decay carries its
    exponential's error, (4 + 2 |g|) U, and a product's rounding U, whatever the order of
    the products; each addition U, at most one per token plus 48 where runs are joined."""
    B, T, D = x.shape
    seqs = sequences(B, T, cu)
    h, bound = np.zeros((B, T, D)), np.zeros((B, T, D))
    final, fbound = np.zeros((len(seqs), D)), np.zeros((len(seqs), D))
    a = np.exp(g)
    with np.errstate(invalid="ignore"):
        f = np.where(np.isinf(g), 0.0, (6 + 2 * np.abs(np.where(np.isinf(g), 0.0, g))) * U)
    for b, n, t0, t1 in seqs:
        s = np.zeros(D) if init is None else init[n].copy()
        m, e = np.abs(s), np.zeros(D)
        for t in range(t0, t1):
            s = a[b, t] * s + x[b, t]
            e = a[b, t] * (e + f[b, t] * m)
            m = a[b, t] * m + np.abs(x[b, t])
            h[b, t], bound[b, t] = s, e + 48 * U * m
        final[n], fbound[n] = s, e + 48 * U * m
    return h, final, bound, fbound


def scan_bwd(g, h, dh, init=None, cu=None, dfinal=None):
    """(dx, dg, dinit) and their bounds, from the stored h (see ``scan``)."""
    B, T, D = h.shape
    seqs = sequences(B, T, cu)
    dx, dg = np.zeros((B, T, D)), np.zeros((B, T, D))
    bx, bg = np.zeros((B, T, D)), np.zeros((B, T, D))
    di, bi = np.zeros((len(seqs), D)), np.zeros((len(seqs), D))
    a = np.exp(g)
    f = np.where(np.isinf(g), 0.0, (6 + 2 * np.abs(np.where(np.isinf(g), 0.0, g))) * U)
    for b, n, t0, t1 in seqs:
        c = np.zeros(D) if dfinal is None else dfinal[n].copy()     # a_{t+1} delta_{t+1}
        m, e = np.abs(c), np.zeros(D)
        for t in range(t1 - 1, t0 - 1, -1):
            d = dh[b, t] + c
            m = m + np.abs(dh[b, t])
            before = h[b, t - 1] if t > t0 else np.zeros(D) if init is None else init[n]
            dx[b, t], bx[b, t] = d, e + 48 * U * m
            dg[b, t] = d * a[b, t] * before
            bg[b, t] = a[b, t] * np.abs(before) * (bx[b, t] + (f[b, t] + 2 * U) * m)
            c = a[b, t] * d
            e = a[b, t] * (e + f[b, t] * m)
            m = a[b, t] * m
        di[n], bi[n] = c, e + 48 * U * m
    return (dx, dg, di), (bx, bg, bi)


# ---- norms around a block ------------------------------------------------------

def act(z, kind):
    s, one_less = 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z))       # and 1 - s
    return (z * s, s * (1.0 + z * one_less)) if kind == "silu" else (s, s * one_less)


def _chain(y, w, z, kind, r, s, eps):
    rstd1 = 1.0 / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
    y1 = y * rstd1 * w if w is not None else y
    a, da = act(z, kind) if z is not None else (np.ones(()), np.zeros(()))
    y2 = y1 * a
    rp = None if r is None else r + (y2 if s is None else s * y2)
    return rstd1, y1, a, da, y2, rp


def norm(y, w=None, z=None, kind="silu", r=None, s=None, nw=None, eps=1e-6):
    """((out, residual_out), (their bounds)); None where there is none.

    Counts: a row sum adds each element with at most d / 64 + 32 roundings on its way; the
    reciprocal root, its products and the activation 16 more."""
    d = y.shape[-1]
    K = d / 64 + 48
    rstd1, y1, a, da, y2, rp = _chain(y, w, z, kind, r, s, eps)
    b2 = K * U * np.abs(y2)
    if z is not None:
        # the sigmoid's exponential carries |z| U more; silu's and sigmoid's relative error alike
        b2 = b2 + 2 * np.abs(z) * U * np.abs(y2)
    if r is None:
        return (y2, None), (b2, None)
    br = (np.abs(s) if s is not None else 1.0) * (b2 + 2 * U * np.abs(y2)) + 2 * U * np.abs(rp)
    if nw is None:
        return (None, rp), (None, br)
    q = (rp * rp).mean(-1, keepdims=True) + eps
    rstd2 = 1.0 / np.sqrt(q)
    n = rp * rstd2 * nw
    rel = (np.abs(rp) * br).mean(-1, keepdims=True) / q + K * U
    return (n, rp), (np.abs(n) * rel + br * rstd2 * np.abs(nw), br)


def norm_bwd(y, dout, w=None, z=None, kind="silu", r=None, s=None, nw=None, drout=None, eps=1e-6):
    """Gradients as a dict (y, weight, gate, residual, scale, next) and their bounds: the
    formula over magnitudes times the roundings on the longest way (two row sums, the
    activation and its derivative; for the parameters the rows of one partial sum, taken as
    rows / 64 + 256)."""
    d, rows = y.shape[-1], y.size // y.shape[-1] if y.size else 0
    K = (2 * (d / 64 + 32) + 64) * U
    ax = tuple(range(y.ndim - 1))
    rstd1, y1, a, da, y2, rp = _chain(y, w, z, kind, r, s, eps)
    if z is not None:
        K = K * (1 + 0.1 * np.abs(z).max(initial=0.0))
    C = K + (rows / 64 + 256) * U
    out, bnd = {}, {}
    mean = lambda t: t.mean(-1, keepdims=True)
    if r is None:
        dv, mv = dout, np.abs(dout)
    else:
        dv = np.zeros(rp.shape) if drout is None else drout
        mv = np.abs(dv)
        if nw is not None:
            q = mean(rp * rp) + eps
            rstd2 = 1.0 / np.sqrt(q)
            t = dout * nw
            mr = np.abs(r) + np.abs(y2 if s is None else s * y2)      # r' may cancel
            rho = mean(mr * np.abs(rp)) / q + 1.0                    # and its root's error with it
            out["next"] = (dout * rp * rstd2).sum(ax)
            bnd["next"] = C * (rho * np.abs(dout) * mr * rstd2).sum(ax)
            dv = dv + rstd2 * (t - rp * rstd2 ** 2 * mean(t * rp))
            mv = mv + 3 * rho * rstd2 * (np.abs(t) + mr * rstd2 ** 2 * mean(np.abs(t) * mr))
        out["residual"], bnd["residual"] = dv, K * mv
        if s is not None:
            out["scale"], bnd["scale"] = (dv * y2).sum(ax), C * (mv * np.abs(y2)).sum(ax)
            dv, mv = dv * s, mv * np.abs(s)
    if z is not None:
        # act' of silu is a difference that cancels near z = -1.28: its magnitude
        mda = (1.0 + np.abs(z)) / (1.0 + np.exp(-z)) if kind == "silu" else da
        out["gate"], bnd["gate"] = dv * y1 * da, K * mv * np.abs(y1) * mda
        dv, mv = dv * a, mv * np.abs(a)
    if w is not None:
        out["weight"], bnd["weight"] = (dv * y * rstd1).sum(ax), C * (mv * np.abs(y) * rstd1).sum(ax)
        t, mt = dv * w, mv * np.abs(w)
        dv = rstd1 * (t - y * rstd1 ** 2 * mean(t * y))
        mv = 3 * rstd1 * (mt + np.abs(y) * rstd1 ** 2 * mean(mt * np.abs(y)))
    out["y"], bnd["y"] = dv, K * mv
    return out, bnd


# ---- delta rule on a cache of states -------------------------------------------

def delta_step(q, k, v, beta, state, g=None, n_h=1, slots=None):
    """(out, new state) and their bounds.  Requests whose slot is -1, out of range or named
    before in the call leave the state alone and read zeros.

    Counts: a sum over the d_k rows adds with at most 24 roundings on the way."""
    N, T, H, dk = q.shape
    dv = v.shape[-1]
    S, ES = state.astype(np.float64).copy(), np.zeros(state.shape)
    out, bo = np.zeros((N, T, H, dv)), np.zeros((N, T, H, dv))
    seen = set()
    for n in range(N):
        slot = n if slots is None else int(slots[n])
        if slot < 0 or slot >= S.shape[0] or slot in seen:
            continue
        seen.add(slot)
        s, e = S[slot], ES[slot]                                     # [H, dk, dv]
        for t in range(T):
            if g is not None:
                gt = g[n, t][..., None] if g.ndim == 4 else g[n, t][:, None, None]
                e = np.exp(gt) * (e + (6 + 2 * np.abs(gt)) * U * np.abs(s))
                s = np.exp(gt) * s
            for j in range(t * n_h, (t + 1) * n_h):
                kk, b = k[n, j][..., None], beta[n, j][:, None]
                ak = np.abs(kk)
                ks, mks = (kk * s).sum(1), (ak * np.abs(s)).sum(1)
                eks = (ak * e).sum(1) + 24 * U * mks
                u = b * (v[n, j] - ks)
                eu = np.abs(b) * (eks + 2 * U * (np.abs(v[n, j]) + mks)) + U * np.abs(u)
                before, eb = np.abs(s), e
                s = s + kk * u[:, None]
                e = eb + ak * eu[:, None] + 2 * U * (before + ak * np.abs(u)[:, None])
            aq = np.abs(q[n, t])[..., None]
            out[n, t] = (q[n, t][..., None] * s).sum(1)
            bo[n, t] = (aq * e).sum(1) + 48 * U * (aq * (before + ak * np.abs(u)[:, None])).sum(1)
        S[slot], ES[slot] = s, e
    return (out, S), (bo, ES)
