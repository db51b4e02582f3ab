"""Plain 64-bit definitions of the 8-bit-row operators (CPU, numpy), shared by their tests."""
import numpy as np

import datagen


def scale(x, fmt):
    """Scale of each row of the float64 matrix x (values of a 16- or 32-bit type): "e4m3" or "int8"."""
    top = np.max(np.abs(x), axis=-1)
    with np.errstate(all="ignore"):
        if fmt == "e4m3":
            s = np.ones_like(top)
            for i, t in np.ndenumerate(top):
                if np.isfinite(t) and t > 0:
                    m, e = np.frexp(t)  # t = m 2^e, 1/2 <= m < 1; 448 = 7/8 2^9
                    s[i] = 2.0 ** min(max(e - 9 + (m > 0.875), -126), 119)
        else:
            s = (top.astype(np.float32) / np.float32(127)).astype(np.float64)
            s = np.where(top == 0, 1.0, np.clip(s, 2.0 ** -126, 2.0 ** 121))
    return np.where(np.isfinite(top), s, np.nan)


def quantize(x, fmt):
    """(bytes, scale) of the rows of x."""
    s = scale(x, fmt)
    fine = np.isfinite(s)
    xs = np.where(fine[..., None], x, 0.0)
    ss = np.where(fine, s, 1.0)[..., None]
    if fmt == "e4m3":  # a power of two: the quotient is exact in 64 bits
        b = datagen.e4m3_bytes((xs / ss).astype(np.float32))
    else:
        q = (xs.astype(np.float32) / ss.astype(np.float32)).astype(np.float64)
        b = np.clip(np.rint(q), -127, 127).astype(np.int8).view(np.uint8)
    return b.reshape(x.shape), s


def values(b, s, fmt):
    v = datagen.e4m3_decode(b) if fmt == "e4m3" else np.asarray(b).view(np.int8).astype(np.float64)
    return v.reshape(np.shape(b)) * np.asarray(s, np.float64)[..., None]


def sigmoid(g):
    return np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))


def gated(g, u):
    return g * sigmoid(g) * u


def gated_grad(g, u, dh):
    p = sigmoid(g)
    return dh * u * p * (1 + g * (1 - p)), dh * g * p


def pair_places(rot, inter):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)


def turned(v, cos, sin, inter):
    """v [tokens, heads, dim] turned by cos, sin [tokens, rot / 2]."""
    a, b = pair_places(2 * cos.shape[1], inter)
    c, s = cos[:, None], sin[:, None]
    r = v.copy()
    r[..., a] = v[..., a] * c - v[..., b] * s
    r[..., b] = v[..., b] * c + v[..., a] * s
    return r


def head_weights(heads, nq, wq, wk):
    return np.stack([wq if h < nq else wk for h in range(heads)])


def head_norm_rope(x, nq, wq, wk, cos, sin, eps, inter):
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    return turned(x * r * head_weights(x.shape[1], nq, wq, wk), cos, sin, inter)


def head_norm_rope_grad(dy, x, nq, wq, wk, cos, sin, eps, inter):
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    g = turned(dy, cos, -sin, inter)
    d = g * head_weights(x.shape[1], nq, wq, wk)
    dx = r * (d - x * r * np.mean(d * x * r, -1, keepdims=True))
    dw = g * x * r
    return dx, dw[:, :nq].sum((0, 1)), dw[:, nq:].sum((0, 1))
