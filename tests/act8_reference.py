"""Plain 64-bit forms of the feed-forward block's operators, and the error
bounds that their tests allow, for the GPU tests.

Bounds, from the arithmetic (u = 2^-24, half a step of fp32):

* product: (m + 16) u sum over runs |sx sw P|, P the exact sum of a run of
  gcd(group, 128) columns, m the number of runs.  A run brings the rounding of
  its scale and of one addition; the partial sums never exceed the sum of the
  magnitudes, whatever the order; 16 covers the sums over warps and splits.
* silu(g) u: silu' <= 1.1, so 1.1 dg (|u| + du) + |silu(g)| du, and 8 u |h| for
  expf (2 steps, i.e. 4 u), the addition, the division and the product.
* 8-bit form of y: the scale is off by max(dy) / 127 and 2 u of itself; q is
  rint(y inv) with y inv off by 4 u relative, at most 127 * 4 u, so
  |s q - y| <= s / 2 + 127 * 4 u s + dy.
* norm: the mean square is a sum of d positive terms over at least 128
  threads, so it is off by (d / 128 + 16) u relative; the root halves that;
  the mean, root, reciprocal and two products add 8 u.
* a rounding to bf16 adds 2^-8 of the value.
"""
import math

import numpy as np

from oracle import gptq_oracle as O

U = 2.0 ** -24


def weights(words, scales, zeros, group):
    """(s expanded, q - z) of a packed layer, fp64."""
    words = np.asarray(words).view(np.uint32)
    d_col = words.shape[1] * 8
    q = O.unpack_codes(words, 4, d_col).astype(np.float64)
    gi = np.arange(d_col) // (group if group else d_col)
    return np.asarray(scales, np.float64)[:, gi], q - np.asarray(zeros, np.float64)[:, gi]


def activation_scales(x_scales, d):
    """One scale a column."""
    x_scales = np.asarray(x_scales, np.float64)
    if x_scales.shape[1] == 1:
        return np.broadcast_to(x_scales, (x_scales.shape[0], d))
    return x_scales[:, np.arange(d) // 128]


def product(words, scales, zeros, group, codes, x_scales):
    """Y and its bound, fp64."""
    s, v = weights(words, scales, zeros, group)
    codes = np.asarray(codes, np.float64)
    d = codes.shape[1]
    sx = activation_scales(x_scales, d)
    run = math.gcd(group, 128) if group else 128
    y = np.zeros((codes.shape[0], v.shape[0]))
    mag = np.zeros_like(y)
    for k in range(0, d, run):
        e = min(d, k + run)
        term = (codes[:, k:e] @ v[:, k:e].T) * sx[:, k:k + 1] * s[None, :, k]
        y += term
        mag += np.abs(term)
    return y, (-(-d // run) + 16) * U * mag


def gated(gate, up, group, codes, x_scales):
    """H and its bound, fp64."""
    g, dg = product(*gate, group, codes, x_scales)
    u, du = product(*up, group, codes, x_scales)
    with np.errstate(over="ignore"):
        silu = g / (1.0 + np.exp(-g))
    h = silu * u
    return h, 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + 8 * U * np.abs(h)


def norm(x, residual, weight, eps):
    """y and its bound from the inputs' values (fp64 arrays); `residual` is
    already the sum as stored, or None."""
    r = x if residual is None else residual
    d = r.shape[1]
    y = r / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps)
    if weight is not None:
        y = y * weight
    return y, (0.5 * (d / 128 + 16) + 8) * U * np.abs(y)


def groups_of(d, group):
    return np.arange(d) // (group if group else d)


def check_float(got, ref, bound, bf16=False):
    got = np.asarray(got, np.float64)
    assert np.all(np.isfinite(got))
    tol = bound + (2.0 ** -8 * np.abs(ref) if bf16 else 0.0) + 1e-40
    err = np.abs(got - ref)
    assert np.all(err <= tol), f"worst error over bound {np.max(err / tol):.3f}"


def check_codes(codes, scales, ref, bound, group):
    """codes and scales against the values they stand for."""
    codes, scales = np.asarray(codes, np.float64), np.asarray(scales, np.float64)
    n, d = ref.shape
    gi = groups_of(d, group)
    ng = gi[-1] + 1
    assert scales.shape == (n, ng) and np.all(np.isfinite(scales))
    assert np.abs(codes).max(initial=0) <= 127
    top, slack = np.zeros((n, ng)), np.zeros((n, ng))
    for g in range(ng):
        top[:, g] = np.abs(ref[:, gi == g]).max(axis=1)
        slack[:, g] = bound[:, gi == g].max(axis=1)
    assert np.all(np.abs(scales - top / 127) <= slack / 127 + 2 * U * top / 127 + 2.0 ** -149)
    s = scales[:, gi]
    tol = s / 2 + 127 * 4 * U * s + bound + 2.0 ** -149
    err = np.abs(s * codes - ref)
    assert np.all(err <= tol), f"worst error over bound {np.max(err / tol):.3f}"
