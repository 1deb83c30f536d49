"""Plain 64-bit forms of the gated linear recurrence and of layer
normalisation, step by step from their definitions (numpy, no code shared with
the library), and the error bounds that the tests derive from rounding."""
import numpy as np


def sig(x):
    return 1.0 / (1.0 + np.exp(-x))


def softplus(x):
    return np.logaddexp(0.0, x)


def gates(px, lam, decay):
    """px (..., 3, D) float64 -> r, i, x, y, a, b = sqrt(1 - a^2)"""
    r, i, x = sig(px[..., 0, :]), sig(px[..., 1, :]), px[..., 2, :]
    y = decay * softplus(lam) * r
    return r, i, x, y, np.exp(-y), np.sqrt(-np.expm1(-2 * y))


def forward(px, lam, decay, h0=None, reset=None):
    """H (B,T,D) and the last state (B,D)"""
    B, T, _, D = px.shape
    _, i, x, _, a, b = gates(px, lam, decay)
    h = np.zeros((B, D)) if h0 is None else h0.astype(np.float64)
    H = np.zeros((B, T, D))
    for t in range(T):
        if reset is not None:
            h = np.where(reset[:, t, None] != 0, 0.0, h)
        h = a[:, t] * h + b[:, t] * i[:, t] * x[:, t]
        H[:, t] = h
    return H, h


def backward(px, lam, decay, dH, h0=None, reset=None, dlast=None):
    """dpx (B,T,3,D), dlam (D), dh0 (B,D), by the chain rule step by step"""
    B, T, _, D = px.shape
    r, i, x, y, a, b = gates(px, lam, decay)
    H, _ = forward(px, lam, decay, h0, reset)
    dpx = np.zeros(px.shape)
    dlam = np.zeros(D)
    carry = np.zeros((B, D)) if dlast is None else dlast.astype(np.float64)
    for t in range(T - 1, -1, -1):
        prev = H[:, t - 1] if t else (np.zeros((B, D)) if h0 is None else h0.astype(np.float64))
        new = np.zeros((B, 1)) if reset is None else (reset[:, t, None] != 0)
        prev = np.where(new, 0.0, prev)
        l = dH[:, t] + carry
        da = l * (prev - a[:, t] / b[:, t] * i[:, t] * x[:, t])
        dy = -a[:, t] * da
        dpx[:, t, 0] = dy * y[:, t] * (1 - r[:, t])
        dpx[:, t, 1] = l * b[:, t] * x[:, t] * i[:, t] * (1 - i[:, t])
        dpx[:, t, 2] = l * b[:, t] * i[:, t]
        dlam += (dy * r[:, t] * decay * sig(lam)).sum(0)
        carry = np.where(new, 0.0, a[:, t] * l)
    return dpx, dlam, carry


def step(px, lam, decay, state, slots):
    """rows in order; returns (y with NaN in rows of padding, the new state)"""
    state = state.astype(np.float64).copy()
    _, i, x, _, a, b = gates(px, lam, decay)
    y = np.full(i.shape, np.nan)
    for n, s in enumerate(slots):
        if 0 <= s < state.shape[0]:
            state[s] = a[n] * state[s] + b[n] * i[n] * x[n]
            y[n] = state[s]
    return y, state


def norm(x, w, b, eps):
    """x (M,P,N) -> y, mean, rstd"""
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    return (y if w is None else y * w) + (0.0 if b is None else b), mean, rstd


def norm_backward(x, dy, w, eps):
    _, mean, rstd = norm(x, None, None, eps)
    xh = (x - mean[..., None]) * rstd[..., None]
    d = dy if w is None else dy * w
    dx = rstd[..., None] * (d - d.mean(-1, keepdims=True) - xh * (d * xh).mean(-1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


# ---- error bounds -------------------------------------------------------------
# U is float32's half step.  A gate sig(p) comes from an approximate base-2
# exponential and reciprocal: 2^-22 each by their specification, and the rounded
# argument p log2(e) moves the exponential by |p| U relative, below 2^-21 for
# |p| <= 8; SIG = 2^-20 covers the sum.  y = k r adds k's own rounding (a few U),
# and 1 - e^-y, b = sqrt(m (2 - m)) and u = b i x a few U each: GATE = 2^-19.
U = 2.0 ** -24
SIG, GATE = 2.0 ** -20, 2.0 ** -19
HALF = {"f32": U, "bf16": 2.0 ** -8}


def forward_bound(px, lam, decay, dtype, h0=None, reset=None):
    """elementwise bound of |H - forward()| for outputs of `dtype`, and of the
    float32 state: the recursion of the errors beside that of the values.  Per
    step a is off by a y GATE + U, u by GATE |u|, and the step's two roundings by
    2 U |h|.  Joining tiles forms the same values from products of up to T factors:
    each rounding there is one more U of a value that is not larger than the
    largest state so far, counted once more."""
    B, T, _, D = px.shape
    _, i, x, y, a, b = gates(px, lam, decay)
    u = b * i * x
    h = np.zeros((B, D)) if h0 is None else h0.astype(np.float64)
    e = np.zeros((B, D))
    E, big = np.zeros((B, T, D)), np.abs(h)
    for t in range(T):
        if reset is not None:
            new = reset[:, t, None] != 0
            h, e, big = np.where(new, 0.0, h), np.where(new, 0.0, e), np.where(new, 0.0, big)
        hn = a[:, t] * h + u[:, t]
        big = np.maximum(big, np.maximum(np.abs(hn), np.abs(u[:, t])))
        e = a[:, t] * e + (a[:, t] * y[:, t] * GATE + U) * np.abs(h) + GATE * np.abs(u[:, t]) + 4 * U * big
        h = hn
        E[:, t] = e
    H, _ = forward(px, lam, decay, h0, reset)
    return E + (0 if dtype == "f32" else HALF[dtype] * (np.abs(H) + E)), e


def backward_bound(px, lam, decay, dH, dtype, h0=None, reset=None, dlast=None):
    """bounds for dpx, dlam and dh0, from forward_bound's error of h and the same
    recursion for the adjoint"""
    B, T, _, D = px.shape
    r, i, x, y, a, b = gates(px, lam, decay)
    H, _ = forward(px, lam, decay, h0, reset)
    Eh, _ = forward_bound(px, lam, decay, "f32", h0, reset)
    l = np.zeros((B, T, D))
    El = np.zeros((B, T, D))
    c = np.zeros((B, D)) if dlast is None else dlast.astype(np.float64)
    ec, big = np.zeros((B, D)), np.abs(c)
    for t in range(T - 1, -1, -1):
        l[:, t] = dH[:, t] + c
        big = np.maximum(big, np.abs(l[:, t]) + np.abs(dH[:, t]))
        El[:, t] = ec + 4 * U * big
        new = np.zeros((B, 1), bool) if reset is None else reset[:, t, None] != 0
        c = np.where(new, 0.0, a[:, t] * l[:, t])
        ec = np.where(new, 0.0, a[:, t] * El[:, t] + (a[:, t] * y[:, t] * GATE + 2 * U) * np.abs(l[:, t]))
        big = np.where(new, 0.0, big)
    prev = np.concatenate([(np.zeros((B, 1, D)) if h0 is None else h0[:, None].astype(np.float64)), H[:, :-1]], 1)
    eprev = np.concatenate([np.zeros((B, 1, D)), Eh[:, :-1]], 1)
    if reset is not None:
        new = reset[:, :, None] != 0
        prev, eprev = np.where(new, 0.0, prev), np.where(new, 0.0, eprev)
    q1, q2 = a * a / b * i * x, a * prev
    ex = np.abs(b * i) * El + 2 * GATE * np.abs(l * b * i)
    ei = np.abs(x) * ((1 - i) * ex + np.abs(l * b * i) * (SIG * i + 2 * U))
    w = y * l * (q1 - q2)
    ew = y * (np.abs(q1 - q2) * El + np.abs(l) * (a * eprev + 3 * GATE * np.abs(q1) + (GATE * y + 4 * U) * np.abs(q2)))
    ew += 2 * GATE * np.abs(w)
    er = (1 - r) * ew + np.abs(w) * (SIG * r + 2 * U)
    E = np.stack([er, ei, ex], axis=2)
    if dtype != "f32":
        dpx, _, _ = backward(px, lam, decay, dH, h0, reset, dlast)
        E = E + HALF[dtype] * (np.abs(dpx) + E)
    ratio = sig(lam) / softplus(lam)
    # any order of B T additions: at most B T half steps of the sum of magnitudes
    elam = ratio * (ew.sum((0, 1)) + (B * T + 16) * U * np.abs(w).sum((0, 1)))
    return E, elam, ec


def norm_bounds(x, w, b, eps, dtype, dy=None):
    """bounds for y, mean, rstd and, with dy, dx, dweight, dbias.  Sums of n terms
    in any order are off by n U of the sum of magnitudes; rounding one of the
    values by a relative e moves it by e of its own size."""
    M, P, N = x.shape
    y, mean, rstd = norm(x, w, b, eps)
    xc = x - mean[..., None]
    xh = xc * rstd[..., None]
    em = (N + 2) * U * np.abs(x).mean(-1)
    # the sum of squares about a mean that is off by em grows by N em^2
    ev = (N + 6) * U * (xc ** 2).mean(-1) + 2 * U * np.abs(x).max(-1) * np.abs(xc).mean(-1) + em ** 2
    er = rstd * (0.5 * ev * rstd ** 2 * 1.01 + 4 * U)
    exh = rstd[..., None] * (em[..., None] + U * np.abs(xc)) + np.abs(xc) * er[..., None] + 2 * U * np.abs(xh)
    aw = 1.0 if w is None else np.abs(w)
    ey = exh * aw + 2 * U * (np.abs(xh) * aw + (0.0 if b is None else np.abs(b)))
    out = [ey + (0 if dtype == "f32" else HALF[dtype] * (np.abs(y) + ey)), em, er]
    if dy is None:
        return out
    d = dy if w is None else dy * w
    m1 = np.abs(d).mean(-1, keepdims=True)
    m2 = np.abs(d * xh).mean(-1, keepdims=True)
    em1 = (N + 2) * U * m1
    em2 = (N + 4) * U * m2 + (np.abs(d) * exh).mean(-1, keepdims=True)
    dx, _, _ = norm_backward(x, dy, w, eps)
    edx = rstd[..., None] * (4 * U * (np.abs(d) + m1 + np.abs(xh) * m2) + em1 + np.abs(xh) * em2 + exh * m2)
    edx = edx + er[..., None] / rstd[..., None] * np.abs(dx) + 2 * U * np.abs(dx)
    out.append(edx + (0 if dtype == "f32" else HALF[dtype] * (np.abs(dx) + edx)))
    out.append((np.abs(dy) * exh).sum(0) + (M + 2) * U * np.abs(dy * xh).sum(0))
    out.append((M + 2) * U * np.abs(dy).sum(0))
    return out
