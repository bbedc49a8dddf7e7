"""Plain float64 forms of the gated linear recurrence and of the layer norm, with
the error bounds of the kernels (first order, from the number of roundings)."""
import numpy as np

U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}  # half a step of each type
E32 = 2.0 ** -24


def coefficients(gate, kind):
    if kind == "decay":
        return gate, np.ones_like(gate)
    e = np.exp(-np.abs(gate))
    r = 1 / (1 + e)
    return np.where(gate < 0, e * r, r), np.where(gate < 0, r, e * r)


def step_error(gate, kind):
    """Roundings of one token, in half steps of float32.  A decay that is given: the product of the
    decays and the state, two at most, and the join of two pieces.  A sigmoid: the exponent |g| is
    off by half a step of itself, so exp by |g| of them; exp, the sum, the quotient and the product
    by another 12."""
    return np.full_like(gate, 4.0) if kind == "decay" else np.abs(gate) + 16


def scan(x, gate, h0, kind):
    """x, gate [B, T, D]; h0 [B, D] or None.  (h, error of h), both [B, T, D]."""
    a, b = coefficients(gate, kind)
    k = step_error(gate, kind) * E32 * 1.01
    B, T, D = x.shape
    s = np.zeros((B, D)) if h0 is None else np.array(h0, np.float64)
    m, e = np.abs(s), np.zeros((B, D))
    h, err, mag = (np.zeros(x.shape) for _ in range(3))
    for t in range(T):
        s = a[:, t] * s + b[:, t] * x[:, t]
        m = np.abs(a[:, t]) * m + np.abs(b[:, t] * x[:, t])
        e = np.abs(a[:, t]) * e + k[:, t] * m + 2.0 ** -120 * m
        h[:, t], err[:, t], mag[:, t] = s, e, m
    return h, err, mag


def before(h, h0):
    first = np.zeros_like(h[:, :1]) if h0 is None else np.asarray(h0, np.float64)[:, None]
    return np.concatenate([first, h[:, :-1]], 1)


def scan_grad(x, gate, dh, h0, dhT, kind):
    """{name: (gradient, error)} of dx, dgate, dh0, without the rounding of the result."""
    a, b = coefficients(gate, kind)
    k = step_error(gate, kind) * E32 * 1.01
    h, eh, mh = scan(x, gate, h0, kind)
    past, epast = before(h, h0), before(eh, None)
    mpast = before(mh, None if h0 is None else np.abs(h0))
    B, T, D = x.shape
    G, EG, MG = (np.zeros(x.shape) for _ in range(3))
    u = np.zeros((B, D)) if dhT is None else np.array(dhT, np.float64)
    mu, eu = np.abs(u), np.zeros((B, D))
    for t in reversed(range(T)):
        G[:, t] = dh[:, t] + u
        MG[:, t] = np.abs(dh[:, t]) + mu
        EG[:, t] = eu + 2 * E32 * MG[:, t]
        aa = np.abs(a[:, t])
        u, mu, eu = a[:, t] * G[:, t], aa * MG[:, t], aa * EG[:, t] + (k[:, t] + 2.0 ** -120) * aa * MG[:, t]
    out = {"dx": (b * G, b * (EG + k * MG)), "dh0": (u, eu)}
    diff, mdiff = (past, mpast) if kind == "decay" else (past - x, mpast + np.abs(x))
    ab = 1.0 if kind == "decay" else a * b
    out["dgate"] = (G * diff * ab,
                    (EG * mdiff + MG * epast + (3 * k + 4 * E32) * MG * mdiff) * np.abs(ab))
    return out


def layer_norm(x, w, b, eps):
    """x [N, D].  (y, error of y without its rounding, mean, 1 / deviation)."""
    D = x.shape[-1]
    m = x.mean(-1, keepdims=True)
    c = x - m
    var = (c * c).mean(-1, keepdims=True)
    r = 1 / np.sqrt(var + eps)
    n = c * r
    # a sum is at most 64 additions of a thread and a tree of the threads
    f = E32 * (64 + 24)
    dm = f * np.abs(x).mean(-1, keepdims=True)
    dvar = 2 * f * var + dm * dm
    dr = 0.5 * dvar / (var + eps) + 4 * E32  # relative
    dn = r * (dm + E32 * np.abs(c)) + np.abs(n) * (dr + 2 * E32)
    W = np.ones(D) if w is None else w
    y = n * W + (0 if b is None else b)
    err = np.abs(W) * dn + 3 * E32 * (np.abs(n * W) + (0 if b is None else np.abs(b)))
    return y, 1.01 * err, m, r, 1.01 * dm, 1.01 * dr


def layer_norm_grad(s, dy, m, r, w, ds):
    """{name: (gradient, error)} from the statistics as given."""
    f = E32 * (64 + 24)
    c = s - m
    n = c * r
    dn = r * E32 * np.abs(c) + 2 * E32 * np.abs(n)
    g = dy if w is None else dy * w
    mean = lambda z: z.mean(-1, keepdims=True)  # noqa: E731
    dx = r * (g - mean(g) - n * mean(g * n))
    err = np.abs(r) * (6 * E32 * np.abs(g) + f * mean(np.abs(g)) +
                       np.abs(n) * (f + 4 * E32) * mean(np.abs(g * n)) +
                       dn * mean(np.abs(g * n)) + np.abs(n) * mean(np.abs(g) * dn))
    if ds is not None:
        dx = dx + ds
        err = err + E32 * (np.abs(dx) + np.abs(ds))
    rows = E32 * (len(s) + 8)
    return {"dx": (dx, 1.01 * err),
            "dw": ((dy * n).sum(0), 1.01 * (rows * np.abs(dy * n) + np.abs(dy) * dn).sum(0)),
            "db": (dy.sum(0), 1.01 * rows * np.abs(dy).sum(0))}
