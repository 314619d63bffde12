"""fp64 oracle of the per-head norms of queries and keys with the rotation by position, and of its gradients.

A head's row x of d channels at a position with the angles theta:
y = x w / sqrt(mean(x^2) + eps), then each rotated pair (a, b) of channels, (i, i + rotary / 2) or (2i, 2i + 1),
becomes (a cos - b sin, b cos + a sin).  Written with the rotation as a matrix, row by row.
"""

import numpy as np


def rotation(cos, sin, d, interleaved):
    """The d x d matrix that rotates one position's row (cos, sin: [rotary / 2])."""
    half = len(cos)
    R = np.eye(d)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        R[a, a], R[a, b], R[b, a], R[b, b] = cos[i], -sin[i], sin[i], cos[i]
    return R


def norm_rope64(x, w, cos, sin, eps, interleaved):
    """x [T, heads, d], w [d], cos, sin [T, rotary / 2] -> y [T, heads, d]."""
    y = x * w / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return np.stack([y[t] @ rotation(cos[t], sin[t], x.shape[-1], interleaved).T for t in range(x.shape[0])]
                    ) if x.shape[0] else y


def norm_rope64_backward(dy, x, w, cos, sin, eps, interleaved):
    """(dx, dw) of sum(dy * norm_rope64(x, w, ...))."""
    d = x.shape[-1]
    dx, dw = np.zeros_like(x), np.zeros(d)
    for t in range(x.shape[0]):
        u = dy[t] @ rotation(cos[t], sin[t], d, interleaved)  # R^T dy, as rows
        n = np.sqrt((x[t] * x[t]).mean(-1, keepdims=True) + eps)
        dw += (u * x[t] / n).sum(0)
        dx[t] = u * w / n - x[t] * (u * w * x[t]).sum(-1, keepdims=True) / (d * n ** 3)
    return dx, dw
