"""fp64 oracle of the Linear layer and its gradient: numpy on float64, the error function by scipy.  It
shares no code with the CUDA path."""
import numpy as np
from scipy.special import erf, expit


def activation(v, act):
    if act == "gelu":
        return 0.5 * v * (1.0 + erf(v / np.sqrt(2.0)))
    return v * expit(v) if act == "silu" else v


def derivative(v, act):
    if act == "gelu":
        return 0.5 * (1.0 + erf(v / np.sqrt(2.0))) + v * np.exp(-v * v / 2) / np.sqrt(2 * np.pi)
    if act == "silu":
        return expit(v) + v * expit(v) * expit(-v)
    return np.ones_like(v)


def forward(x, w, bias=None, residual=None, act="none"):
    """(y, z): z = x w^T + bias, y = act(z) + residual."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        z = z + bias
    y = activation(z, act)
    return (y if residual is None else y + residual), z


def backward(x, w, z, d_y, act="none"):
    """(dx, dw, db, dz) for z given as it was kept."""
    dz = np.asarray(d_y, np.float64) * (derivative(np.asarray(z, np.float64), act) if act != "none" else 1.0)
    return dz @ np.asarray(w, np.float64), dz.T @ np.asarray(x, np.float64), dz.sum(0), dz
