"""Plain fp64 implementations of the operators around the softmax layers of a
serving step, written from their definitions (numpy, loops), and the inputs of
their tests."""
import numpy as np

from tests import tree_ref


def norm_rope(x, positions, inv_freq, weight=None, eps=1e-6, interleaved=False):
    """x [T, H, d] -> (y, size): the result and |a| + |b| of each element's pair before the turn."""
    T, H, d = x.shape
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * weight
    out, size = y.copy(), np.abs(y)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + len(inv_freq))
        for t, p in enumerate(positions):
            # exact: an fp32 frequency times an integer fits 64 bits of significand
            angle = float(np.fmod(np.longdouble(float(f)) * int(p), 2 * PI))
            c, s = np.cos(angle), np.sin(angle)
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
            size[t, :, a] = size[t, :, b] = np.abs(y[t, :, a]) + np.abs(y[t, :, b])
    return out, size


# pi to the 64 bits of the extended type (on machines where that is a double, angles are taken there)
PI = np.longdouble("3.14159265358979323846264338327950288")
