"""Plain binary64 forms of the row-wise layers (numpy), with the rounding error
that a binary32 evaluation may have, for the GPU tests.

Tolerances.  u = 2^-24 is half a unit of binary32, E(dt) half a unit of the
output type relative to the value (torch.finfo(dt).eps / 2: bf16 2^-8, fp16 2^-11), plus
half its smallest subnormal step.  The bounds are first-order (terms in u^2 are
covered by the factor SLACK):
  * a sum of k terms in any order is off by at most (k - 1) u sum |terms|; where
    the kernels add along a tree of known depth the depth L replaces k;
  * one row of dim <= 2048 * 64 elements is added along a path of at most L = 48
    additions: 7 within a unit of 8, up to 16 units per thread, 6 steps within a
    wave, 4 between waves, and the second sum's correction.
"""
import numpy as np
import torch

U = 2.0 ** -24
L = 48
SLACK = 1.001


def half_step(dt, y):
    """Half a step of dtype dt at the values y."""
    fi = torch.finfo(dt)
    return fi.eps / 2 * np.abs(y) + fi.smallest_normal * fi.eps / 2


def f64(t):
    return t.detach().cpu().double().numpy()


def statistics(x, eps):
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    return mean, var, 1.0 / np.sqrt(var + eps)


def normalized(x, eps, exact):
    """h = (x - mean) * rstd, mean, rstd, and the kernels' errors of h, mean and rstd.

    exact (binary32 rows): the mean is corrected by the mean of the rounded
    differences d, so it is off by its own rounding u |mean| and by the error
    (L + 2) u mean|x - mean| of that correction (mean|x - mean| <= sqrt(var)).
    Otherwise (16-bit rows) it is the sum's, off by e = (L + 2) u mean|x|.  The
    squared deviations of a row's waves, taken around such means, are joined as
    if these were exact: off by 2 e |d_w| + e^2 for a wave whose mean lies d_w from the
    row's, and the mean of |d_w| over the waves is at most sqrt(var).
    var is off by (L + 6) u relative besides, rstd by half of all that and by 3 u of
    the hardware's reciprocal root (1 ulp = 2 u) and its argument; the
    difference and the product of h round once each."""
    mean, var, rstd = statistics(x, eps)
    h = (x - mean[:, None]) * rstd[:, None]
    if exact:
        e_mean = U * np.abs(mean) + (L + 2) * U * np.sqrt(var)
        e_rel = np.full_like(mean, ((L + 6) / 2 + 3) * U)
    else:
        e_mean = (L + 2) * U * np.abs(x).mean(1)
        e_rel = ((L + 6) / 2 + 3) * U + e_mean * rstd + (e_mean * rstd) ** 2 / 2
    e_h = (e_mean * rstd)[:, None] + np.abs(h) * (e_rel[:, None] + 2 * U)
    return h, mean, rstd, e_h, e_mean, e_rel * rstd


def layer_norm(x, gamma, beta, eps, exact):
    """y, the error of the kernels' binary32 y, and the statistics with theirs."""
    h, mean, rstd, e_h, e_mean, e_rstd = normalized(x, eps, exact)
    g = np.ones(x.shape[1]) if gamma is None else gamma
    b = np.zeros(x.shape[1]) if beta is None else beta
    y = h * g + b
    return y, e_h * np.abs(g) + U * np.abs(y), mean, rstd, e_mean, e_rstd


def norm_grad(dy, e_dy, h, e_h, rstd, e_rstd, gamma):
    """dx of one layer norm and its error, from dy and h that are themselves off
    by e_dy and e_h (rstd by e_rstd)."""
    r = rstd[:, None]
    g = dy * gamma
    e_g = e_dy * np.abs(gamma) + U * np.abs(g)
    ag = np.abs(g) + e_g
    c1, c2 = g.mean(1, keepdims=True), (g * h).mean(1, keepdims=True)
    e_c1 = e_g.mean(1, keepdims=True) + (L + 2) * U * ag.mean(1, keepdims=True)
    agh = (ag * (np.abs(h) + e_h)).mean(1, keepdims=True)
    e_c2 = (e_g * np.abs(h) + np.abs(g) * e_h).mean(1, keepdims=True) + (L + 3) * U * agh
    inner = g - c1 - h * c2
    e_inner = e_g + e_c1 + e_h * np.abs(c2) + np.abs(h) * e_c2 + 3 * U * (ag + np.abs(c1) + np.abs(h * c2))
    dx = r * inner
    return dx, r * e_inner + e_rstd[:, None] * np.abs(inner) + U * np.abs(dx)


def token_sums(dy, ids, rows):
    """S[v] = sum of dy over the tokens of v, and its error (k terms: k u sum |dy|)."""
    s, a, k = np.zeros((rows, dy.shape[1])), np.zeros((rows, dy.shape[1])), np.zeros(rows)
    for t, v in enumerate(ids):
        if 0 <= v < rows:
            s[v] += dy[t]
            a[v] += np.abs(dy[t])
            k[v] += 1
    return s, a * k[:, None] * U, k


def column_sum(terms, e_terms):
    """Sum over the rows and its error: at most min(n, 128) + 8 additions on a path."""
    k = min(terms.shape[0], 128) + 8
    return terms.sum(0), e_terms.sum(0) + k * U * (np.abs(terms) + e_terms).sum(0)


def assert_close(got, want, err, what):
    """|got - want| <= err * SLACK + half a step of got's dtype, NaN and infinities alike."""
    y = f64(got).reshape(want.shape)
    bound = err * SLACK + half_step(got.dtype, np.abs(want) + err)
    bad = ~(np.abs(y - want) <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(y - want) / np.maximum(bound, 1e-300), 0)), y.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside the bound; at {i} got {y[i]!r}, "
                             f"want {want[i]!r}, bound {bound[i]!r}")
