"""fp64 CPU statement of the activation operators (numpy, no code shared with
the package): 8-bit block-scaled activations, the root-mean-square norm and
its gradient, weight gradients, tokens by expert and back."""
import numpy as np

BLOCK = 32
TOP = {"e4m3": 448.0, "int8": 127.0}


def act8_exponent(amax, fmt):
    """Least k >= -120 with amax <= TOP 2^k, for an array of finite maxima."""
    amax = np.asarray(amax, np.float64)
    m, e = np.frexp(amax / TOP[fmt])        # amax / TOP = m 2^e, m in [1/2, 1); the division by 448 or 127
    k = np.where(m > 0.5, e, e - 1)         # may round, so the choice is checked with exact products
    k = np.where(amax > TOP[fmt] * np.ldexp(1.0, k), k + 1, k)
    k = np.where(amax <= TOP[fmt] * np.ldexp(1.0, k - 1), k - 1, k)
    return np.maximum(np.where(amax > 0, k, -120), -120).astype(np.int64)


def e4m3_values():
    """The values of the 256 e4m3 codes."""
    v = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (1 + f / 8.0) * 2.0 ** (e - 7)
        v[c] = np.nan if c & 127 == 127 else (-x if c & 128 else x)
    return v


def act8_round(v, fmt):
    """|v| <= TOP to the nearest value of the format, ties to even."""
    if fmt == "int8":
        return np.rint(v)
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e, -5) - 4)
    return np.rint(v / step) * step


def act8(x, fmt):
    """(values, scale bytes) of rows x [T, D] kept in 8 bits."""
    x = np.asarray(x, np.float64)
    T, D = x.shape
    nb = -(-D // BLOCK)
    xb = np.zeros((T, nb * BLOCK))
    xb[:, :D] = x
    xb = xb.reshape(T, nb, BLOCK)
    fine = np.isfinite(xb).all(axis=2)
    xb = np.where(fine[..., None], xb, 0.0)
    k = act8_exponent(np.abs(xb).max(axis=2), fmt)
    v = np.ldexp(act8_round(np.ldexp(xb, -k[..., None]), fmt), k[..., None])
    v = np.where(fine[..., None], v, np.nan)
    return v.reshape(T, nb * BLOCK)[:, :D], np.where(fine, k + 127, 255).astype(np.uint8)


def act8_values(q, scale, D, fmt):
    """Values of stored codes [T, >= D] and scale bytes."""
    q = np.asarray(q)[:, :D]
    v = e4m3_values()[q] if fmt == "e4m3" else q.astype(np.uint8).view(np.int8).astype(np.float64)
    s = np.asarray(scale)[:, np.arange(D) // BLOCK].astype(np.int64)
    return np.where(s == 255, np.nan, v * np.ldexp(1.0, np.where(s == 255, 127, s) - 127))


def rms_norm(h, w, eps):
    """(y, rstd) of rows h [T, D]."""
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * w, rstd


def rms_norm_backward(dy, h, w, rstd, dh=None):
    xhat = h * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - xhat * (g * xhat).mean(axis=1, keepdims=True))
    return (dx if dh is None else dx + dh), (dy * xhat).sum(axis=0)


def weight_grad(dy, x):
    return dy.T @ x


def expert_sort(idx, E):
    """(offsets, source, position), pair by pair."""
    T, K = idx.shape
    rows = [[] for _ in range(E)]
    for p, e in enumerate(idx.reshape(-1).tolist()):
        if 0 <= e < E:
            rows[e].append(p)
    offsets = np.concatenate([[0], np.cumsum([len(r) for r in rows])]).astype(np.int64)
    order = [p for r in rows for p in r]
    source = np.full(T * K, -1, np.int64)
    source[:len(order)] = order
    position = np.full(T * K, -1, np.int64)
    for r, p in enumerate(order):
        position[p] = r
    return offsets, source, position.reshape(T, K)


def expert_combine(y, position, weights):
    T, K = position.shape
    out = np.zeros((T, y.shape[1]))
    for t in range(T):
        for k in range(K):
            if position[t, k] >= 0:
                out[t] += weights[t, k] * y[position[t, k]]
    return out


def expert_combine_backward(dout, y, position, weights, dy):
    """dy is the buffer whose unreached rows stay."""
    T, K = position.shape
    dy, dw = dy.copy(), np.zeros((T, K))
    for t in range(T):
        for k in range(K):
            r = position[t, k]
            if r >= 0:
                dy[r] = weights[t, k] * dout[t]
                dw[t, k] = dout[t] @ y[r]
    return dy, dw


def expert_weight_grad(dy, x, offsets):
    """x in sorted rows, like dy."""
    return np.stack([dy[a:b].T @ x[a:b] for a, b in zip(offsets[:-1], offsets[1:])])
