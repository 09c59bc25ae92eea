"""fp64 oracle of the optimizer step: the global gradient norm, AdamW, and its 8-bit states.

Plain numpy on float64, one tensor at a time; it shares no code with the CUDA path."""
import numpy as np

BLOCK = 256


def e4m3_values():
    """The value of each of the 256 e4m3 codes: 4 exponent bits (bias 7), 3 mantissa bits, no
    infinities, NaN where all seven bits are set."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = np.nan if (c & 127) == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[c] = -v if c & 128 else v
    return out


def grad_norm(grads):
    """sqrt of the sum of squares over every element of every gradient."""
    return np.sqrt(sum(float(np.sum(np.asarray(g, dtype=np.float64) ** 2)) for g in grads))


def block_scale(top):
    """Smallest power of two s >= 2^-126 with top / s <= 448; 0 for top = 0."""
    if top == 0:
        return 0.0
    e = -126
    while top / 2.0 ** e > 448:
        e += 1
    return 2.0 ** e


def block_scales(values):
    """The scale of each block of BLOCK values."""
    v = np.abs(np.asarray(values, dtype=np.float64))
    return np.array([block_scale(v[i:i + BLOCK].max()) for i in range(0, len(v), BLOCK)])


def decode(codes, scales):
    """The values that codes and their blocks' scales stand for."""
    return e4m3_values()[codes] * np.repeat(scales, BLOCK)[:len(codes)]


def adamw(p, g, m, v, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, decay=0.0, norm=None, max_norm=0.0):
    """One step: (parameters, first moments, second moments) after it."""
    p, g, m, v = (np.asarray(a, dtype=np.float64) for a in (p, g, m, v))
    if norm is not None and max_norm > 0 and norm > max_norm:
        g = g * (max_norm / norm)
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    m_hat, v_hat = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p - lr * decay * p - lr * m_hat / (np.sqrt(v_hat) + eps), m, v
