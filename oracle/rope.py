"""The heads' norm and rotation in fp64 numpy, and their gradient, written from the
definition (include/attn_rope.h): one head row after the other, one pair after the
other.  Test infrastructure only."""
import numpy as np


def turn_rows(z, positions, inv_freq, axis, interleaved, back=False):
    """z [B, S, H, D] with its pairs turned by positions [B, S, axes] (back: by the
    negative angles)."""
    z = np.array(z, np.float64)
    n = len(inv_freq)
    for i in range(n):
        a = positions[:, :, axis[i]].astype(np.float64) * inv_freq[i]
        if back:
            a = -a
        c, s = np.cos(a)[:, :, None], np.sin(a)[:, :, None]
        u, w = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        x, y = z[..., u].copy(), z[..., w].copy()
        z[..., u] = x * c - y * s
        z[..., w] = x * s + y * c
    return z


def rope_fwd(x, weight=None, positions=None, inv_freq=(), axis=None, interleaved=False, eps=1e-6):
    """y [B, H, S, D] of one part x [B, S, H, D]."""
    x = np.asarray(x, np.float64)
    z = x
    if weight is not None:
        z = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if len(inv_freq):
        z = turn_rows(z, positions, inv_freq, axis if axis is not None else [0] * len(inv_freq), interleaved)
    return np.ascontiguousarray(z.transpose(0, 2, 1, 3))


def rope_bwd(dy, x, weight=None, positions=None, inv_freq=(), axis=None, interleaved=False, eps=1e-6):
    """dx [B, S, H, D] and dweight [D] (None without weight) for dy [B, H, S, D]; and the
    magnitudes their sums go over, for bounds on rounding: of dx and of dweight."""
    dz = np.asarray(dy, np.float64).transpose(0, 2, 1, 3)
    mag = np.abs(dz)
    if len(inv_freq):
        ax = axis if axis is not None else [0] * len(inv_freq)
        dz = turn_rows(dz, positions, inv_freq, ax, interleaved, back=True)
        n = len(inv_freq)
        mag = mag.copy()
        for i in range(n):
            u, w = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            mag[..., u] = mag[..., w] = mag[..., u] + mag[..., w]
    if weight is None:
        return dz, None, mag, None
    x, weight = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    unit = x * r
    g = dz * weight
    dx = r * (g - unit * (g * unit).mean(-1, keepdims=True))
    m = mag * np.abs(weight)
    dx_mag = r * (m + np.abs(unit) * (m * np.abs(unit)).mean(-1, keepdims=True))
    return dx, (dz * unit).sum((0, 1, 2)), dx_mag, (mag * np.abs(unit)).sum((0, 1, 2))
