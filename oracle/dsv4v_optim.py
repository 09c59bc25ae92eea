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


# ---------------------------------------------------------------------------------------------- stochastic rounding
def philox(counter, key, rounds=7):
    """Philox 4x32 (Salmon, Moraes, Dror and Shaw, 2011): four arrays of 32-bit words from four counter words and two
    key words."""
    c, k, low = [np.asarray(x, dtype=np.uint64) for x in counter], [int(x) for x in key], np.uint64(0xFFFFFFFF)
    for _ in range(rounds):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def draws(n, step, tensor):
    """Uniform numbers in [0, 1) of n elements of a tensor at a step: (first moment's, second moment's)."""
    pairs = (n + 1) // 2
    group, call = np.arange(pairs) // 4, np.arange(pairs) % 4
    w = philox([group & 0xFFFFFFFF, (group >> 32) * 4 + call, np.full(pairs, step & 0xFFFFFFFF), np.full(pairs, step >> 32)], (tensor, 0))
    u = [(x >> np.uint64(8)).astype(np.float64) * 2.0 ** -24 for x in w]
    return np.stack([u[0], u[2]], 1).reshape(-1)[:n], np.stack([u[1], u[3]], 1).reshape(-1)[:n]


def code_neighbours(q):
    """The e4m3 values at or below and above q >= 0 (the next one where q is a value itself)."""
    values = e4m3_values()[:127]
    at = np.searchsorted(values, q, side="right") - 1
    return values[at], np.append(values, 480.0)[at + 1]


def stochastic_codes(m, v, step, tensor):
    """(scaled first moments, scaled roots, scales of each) as values of codes: rounded so that the expectations of the
    first moment and of the root's square are kept; a root above zero is at least the smallest code."""
    m, v = np.asarray(m, dtype=np.float64), np.asarray(v, dtype=np.float64)
    um, uv = draws(len(m), step, tensor)
    sm, sr = block_scales(m), block_scales(np.sqrt(v))
    each = lambda s: np.repeat(np.where(s > 0, s, 1.0), BLOCK)[:len(m)]  # noqa: E731
    q = np.abs(m) / each(sm)
    lo, hi = code_neighbours(q)
    qm = np.copysign(np.minimum(np.where(um < (q - lo) / (hi - lo), hi, lo), 448.0), m)
    x = v / each(sr) ** 2
    lo, hi = code_neighbours(np.sqrt(x))
    qr = np.minimum(np.where(uv < (x - lo * lo) / (hi * hi - lo * lo), hi, lo), 448.0)
    return qm, np.where(v > 0, np.maximum(qr, 2.0 ** -9), 0.0), sm, sr
