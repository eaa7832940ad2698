"""fp64 reference of rotary positions — TEST INFRASTRUCTURE ONLY.

Pair p of a head's first ``rot`` elements turns by the angle
a = positions[axis of p] * inv_freq[p]:

    (x, y) -> (x cos a - y sin a, y cos a + x sin a),

pair p being elements (p, p + rot/2), or (2p, 2p + 1) when interleaved; the
elements from ``rot`` on pass through.  The rotation is orthogonal, so its
backward pass is the rotation by -a.
"""

import numpy as np


def rope_rotate(x, positions, inv_freq, pair_axis=None, interleaved=False, inverse=False):
    """x [..., n, d] rotated by positions [n] or [axes, n] (int), inv_freq
    [rot/2] taken as the exact values given, pair_axis [rot/2] ints.  Returns
    fp64."""
    x = np.asarray(x, dtype=np.float64)
    pos = np.atleast_2d(np.asarray(positions)).astype(np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    half = f.shape[0]
    axis = np.zeros(half, dtype=np.int64) if pair_axis is None else np.asarray(pair_axis)
    out = x.copy()
    for p in range(half):
        a = pos[axis[p]] * f[p] * (-1.0 if inverse else 1.0)
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        out[..., i] = x[..., i] * np.cos(a) - x[..., j] * np.sin(a)
        out[..., j] = x[..., j] * np.cos(a) + x[..., i] * np.sin(a)
    return out
