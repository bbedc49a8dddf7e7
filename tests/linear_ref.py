"""Plain float64 forms of the norm with rotation and of linear attention with a
decay for each head, token by token, and the error bounds of the kernels."""
import numpy as np

U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}  # half a step of each type


def linear(q, k, v, a, S0=None, scale=1.0):
    """q, k [B, T, Hq, K]; v [B, T, H, V]; a [H]; S0 [B, H, V, K].  (o, S_T)."""
    B, T, H, V = v.shape
    g = H // q.shape[2]
    q, k = np.repeat(q, g, 2), np.repeat(k, g, 2)
    S = np.zeros((B, H, V, k.shape[3])) if S0 is None else np.array(S0, np.float64)
    o = np.zeros(v.shape)
    for t in range(T):
        S = a[:, None, None] * S + v[:, t, :, :, None] * k[:, t, :, None, :]
        o[:, t] = scale * np.einsum("bhvk,bhk->bhv", S, q[:, t])
    return o, S


def linear_grad(q, k, v, a, do, S0=None, dST=None, scale=1.0):
    """(dq, dk, dv, dS0) by the adjoint recurrence, with the states kept."""
    B, T, H, V = v.shape
    Hq, K = q.shape[2:]
    g = H // Hq
    qr, kr = np.repeat(q, g, 2), np.repeat(k, g, 2)
    S = np.zeros((B, H, V, K)) if S0 is None else np.array(S0, np.float64)
    states = []
    for t in range(T):
        S = a[:, None, None] * S + v[:, t, :, :, None] * kr[:, t, :, None, :]
        states.append(S)
    R = np.zeros((B, H, V, K)) if dST is None else np.array(dST, np.float64)
    dq, dk, dv = np.zeros((B, T, H, K)), np.zeros((B, T, H, K)), np.zeros((B, T, H, V))
    for t in reversed(range(T)):
        R = R + scale * do[:, t, :, :, None] * qr[:, t, :, None, :]
        dq[:, t] = scale * np.einsum("bhvk,bhv->bhk", states[t], do[:, t])
        dk[:, t] = np.einsum("bhvk,bhv->bhk", R, v[:, t])
        dv[:, t] = np.einsum("bhvk,bhk->bhv", R, kr[:, t])
        R = a[:, None, None] * R
    dq, dk = (x.reshape(B, T, Hq, g, K).sum(3) for x in (dq, dk))
    return dq, dk, dv, R


def steps(dtype, T, width):
    """Relative error of a sum of products over T tokens and `width` channels,
    against the sum of the products' magnitudes: one rounding of an operand in
    bf16 runs, and one float32 step (the tensor cores may cut where the CUDA
    cores round: 2^-23) for each addition, the decay powers' included."""
    f = 2.0 ** -23 * (T + width + 64)
    return f if dtype == "fp32" else U["bf16"] * 1.01 + f


def state_steps(dtype, T):
    """The same for a state: bf16 runs split the weighted operand in two, so
    that what is left of it is U^2."""
    f = 2.0 ** -23 * (T + 64)
    return f if dtype == "fp32" else U["bf16"] ** 2 * 1.01 + f


def norm_rotate(x, w, pos, inv_freq, norm, pairing, eps):
    """x [..., h, D] with pos [...]."""
    x = np.asarray(x, np.float64)
    D, R = x.shape[-1], 2 * len(inv_freq)
    ss = (x * x).sum(-1, keepdims=True)
    y = x / np.sqrt((ss / D if norm == "rms" else ss) + eps)
    if w is not None:
        y = y * np.asarray(w, np.float64)
    ang = (pos[..., None].astype(np.float64) * np.asarray(inv_freq, np.float64))[..., None, :]
    c, s = np.cos(ang), np.sin(ang)
    i = np.arange(R // 2)
    a, b = (i, i + R // 2) if pairing == "half" else (2 * i, 2 * i + 1)
    out = y.copy()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., a] * s + y[..., b] * c
    return out


def norm_rotate_grad(x, w, pos, inv_freq, dy, norm, pairing, eps):
    """(dx, dw)."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    D, R = x.shape[-1], 2 * len(inv_freq)
    ang = (pos[..., None].astype(np.float64) * np.asarray(inv_freq, np.float64))[..., None, :]
    c, s = np.cos(ang), np.sin(ang)
    i = np.arange(R // 2)
    a, b = (i, i + R // 2) if pairing == "half" else (2 * i, 2 * i + 1)
    g = dy.copy()
    g[..., a] = dy[..., a] * c + dy[..., b] * s
    g[..., b] = dy[..., b] * c - dy[..., a] * s
    cn = 1 / D if norm == "rms" else 1.0
    r = 1 / np.sqrt(cn * (x * x).sum(-1, keepdims=True) + eps)
    dw = (g * x * r).reshape(-1, D).sum(0)
    h = g if w is None else g * np.asarray(w, np.float64)
    return r * (h - cn * r * r * x * (x * h).sum(-1, keepdims=True)), dw
