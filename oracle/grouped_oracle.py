"""Products by expert, their gradients and MX FP4 in fp64 numpy, written from
the definitions alone."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def grouped_matmul(x, w, offsets, out, bias=None):
    """out[r] = x[r] @ w[e] (+ bias[e]) for the rows of each expert; other
    rows keep what `out` holds."""
    y = np.array(out, dtype=np.float64)
    for e in range(len(offsets) - 1):
        rows = slice(offsets[e], offsets[e + 1])
        y[rows] = x[rows] @ w[e] + (0.0 if bias is None else bias[e])
    return y


def grouped_weight_grad(x, dy, offsets):
    return np.stack([x[a:b].T @ dy[a:b] for a, b in zip(offsets, offsets[1:])])


def swiglu(gate_up, weights=None):
    g, u = np.split(np.asarray(gate_up, np.float64), 2, axis=1)
    with np.errstate(over="ignore"):
        z = g / (1 + np.exp(-g)) * u
    return z if weights is None else z * weights[:, None]


def swiglu_backward(dz, gate_up, weights=None):
    """(d gate_up, d weights) of swiglu."""
    g, u = np.split(np.asarray(gate_up, np.float64), 2, axis=1)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-g))
    dw = (dz * g * s * u).sum(1)
    if weights is not None:
        dz = dz * weights[:, None]
    return np.concatenate([dz * u * (s + g * s * (1 - s)), dz * g * s], axis=1), dw


def quant_mx_fp4(z):
    """(codes [M, K] of 4 bits, scales [M, K/32]) of finite z: by distance to
    the E2M1 values, the even code where two are as near."""
    M, K = z.shape
    b = z.reshape(M, K // 32, 32)
    amax = np.abs(b).max(2)
    _, e = np.frexp(amax)                       # amax = m 2^e, m in [0.5, 1)
    scale = np.where(amax > 0, np.maximum(e - 1 - 2 + 127, 0), 0)
    v = np.ldexp(b, (127 - scale)[..., None])
    d = np.abs(np.abs(v)[..., None] - E2M1)
    near = d == d.min(-1, keepdims=True)
    order = np.where(np.arange(8) % 2 == 0, 0, 1) + np.where(near, 0, 8)
    code = order.argmin(-1) + 8 * np.signbit(v)
    return code.reshape(M, K), scale


def pack_fp4(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def mx_fp4_values(q4, scale):
    """Values of packed codes [..., K/2] with scales [..., K/32]."""
    q4 = np.asarray(q4).astype(np.int64)
    c = np.stack([q4 & 15, q4 >> 4], -1).reshape(*q4.shape[:-1], -1)
    v = E2M1[c & 7] * np.where(c >= 8, -1.0, 1.0)
    s = np.ldexp(1.0, np.asarray(scale).astype(np.int64) - 127)
    return v * np.repeat(s, 32, axis=-1)


__all__ = ["grouped_matmul", "grouped_weight_grad", "swiglu", "swiglu_backward", "quant_mx_fp4",
           "pack_fp4", "mx_fp4_values"]
