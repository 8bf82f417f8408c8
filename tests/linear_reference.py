"""Plain binary64 forms of the 4-bit layers (numpy), with the rounding error that their
evaluation may have, for the GPU tests.

Tolerances.  u = 2^-24, and E(dt, y) half a step of the output type at y.
  * A sum of k products of two xdt values (exact in binary32 for 16-bit types, one rounding
    each for binary32) in any order is off by at most (k + 2) 2u sum |terms|, which also
    covers matrix instructions that truncate instead of rounding.
  * exp, reciprocal and erfc of the device are off by 1, 1 and 16 units (2u each) at most; an
    argument off by a relative d moves e^x by |x| d and erfc(z / sqrt 2) by at most (z^2 + 1) d
    relative.  With a handful of roundings besides, act(z) is off by at most
    2u (24 + 4 z^2) |act(z)| for gelu and 2u (12 + 4 |q|) |act(z)| for the forms of a
    sigmoid of q (q = z or gelu_tanh's argument, whose own relative error is 4u), and its
    derivative by the same factor times the sum of its terms' absolute values.  An error e of z
    moves act(z) by at most 1.13 e + e^2 (the largest slopes, and the largest curvature 1.2
    halved).  Results below 2^-120 may come out as 0.
  * dz is rounded to the compute dtype before the product: independent errors of at most
    E(dt, dz) each, so that a sum of them exceeds 7 times its root sum of squares with
    probability below 2 e^(-49/2) = 5e-11 (Hoeffding), and never their plain sum.
"""
import numpy as np
import torch

import oracle
from gpu_helpers import DEV, TORCH_DT

U = 2.0 ** -24
DT_OF = {v: k for k, v in TORCH_DT.items()}


def half_step(dt, y):
    fi = torch.finfo(dt)
    return fi.eps / 2 * np.abs(y) + fi.smallest_normal * fi.eps / 2


def f64(t):
    return t.detach().cpu().double().numpy()


class Weight:
    """A random 4-bit weight [n, k]: device arrays, and the values of the compute dtype by the oracle."""

    def __init__(self, n, k, code, blocksize, nested, xdt, seed, blocksize2=256):
        rng = np.random.default_rng(seed)
        nb = -(-n * k // blocksize)
        codes = rng.integers(0, 256, n * k // 2, dtype=np.uint8)
        self.n, self.k, self.code, self.blocksize, self.blocksize2 = n, k, code, blocksize, blocksize2
        self.codes = torch.from_numpy(codes).to(DEV)
        self.absmax = self.dq_parts = None
        if nested:
            c2 = rng.integers(0, 256, nb, dtype=np.uint8)
            a2 = (rng.random(-(-nb // blocksize2)) * 0.02 + 0.005).astype(np.float32)
            mu = np.float32(0.03)
            scale = oracle.dq_decode(c2, a2, mu, blocksize2)
            self.dq_parts = [torch.from_numpy(c2).to(DEV), torch.from_numpy(a2).to(DEV), torch.tensor([mu], device=DEV)]
        else:
            scale = (rng.random(nb) * 0.1 + 0.005).astype(np.float32)
            self.absmax = torch.from_numpy(scale).to(DEV)
        w = oracle.dequantize_blockwise(codes, scale, code, blocksize, n * k, ydt=DT_OF[xdt])
        t = torch.from_numpy(w) if xdt == torch.float32 else torch.from_numpy(w.view(np.int16)).view(xdt)
        self.values = t.view(n, k)
        self.w = self.values.double().numpy()

    def dq(self, L):
        return None if self.dq_parts is None else L.make_dq(*self.dq_parts, self.blocksize2)

    def parts(self, L):
        return self.codes, self.absmax, self.dq(L)


def normal(shape, seed, std=1.0, dtype=torch.float32):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


GELU_A = 2.0 * np.sqrt(2.0 / np.pi)


def act(L, kind, z):
    """act(z), act'(z) and the error of their evaluation."""
    tiny = 2.0 ** -120
    zero = np.zeros_like(z)
    if kind == L.QB_ACT_NONE:
        return z, np.ones_like(z), zero, zero
    if kind == L.QB_ACT_RELU:
        return np.maximum(z, 0.0), (z > 0).astype(float), zero, zero
    if kind == L.QB_ACT_GELU:
        cdf = torch.special.ndtr(torch.from_numpy(np.ascontiguousarray(z))).numpy()
        zp = z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
        rel = 2 * U * (24 + 4 * z * z)
        return z * cdf, cdf + zp, rel * np.abs(z * cdf) + tiny, rel * (cdf + np.abs(zp)) + tiny
    if kind == L.QB_ACT_GELU_TANH:
        q, dq = GELU_A * (z + 0.044715 * z ** 3), GELU_A * (1 + 3 * 0.044715 * z * z)
    else:
        q, dq = z, 1.0
    s, sn = sigmoid(q), sigmoid(-q)
    rel = 2 * U * (12 + 4 * np.abs(q))
    return z * s, s + z * dq * s * sn, rel * np.abs(z * s) + tiny, rel * (s + np.abs(z * dq * s * sn)) + tiny


def assert_close(got, want, err, what):
    """got: a tensor; err: what its binary32 evaluation may be off by before its last rounding."""
    g = f64(got)
    assert g.shape == want.shape, what
    bound = 1.001 * (err + half_step(got.dtype, np.abs(want) + err))
    bad = ~(np.abs(g - want) <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} beyond the bound, first at {np.argwhere(bad)[0]}: "
                           f"{g[bad][0]} for {want[bad][0]} +- {bound[bad][0]}")


def product(x, w):
    """x w^T and its error."""
    return x @ w.T, (x.shape[1] + 2) * 2 * U * (np.abs(x) @ np.abs(w).T)


def linear(L, x, w, bias, kind, residual):
    """(z, its error, y, its error)."""
    z, e = product(x, w)
    if bias is not None:
        z = z + bias
        e = e + U * (np.abs(z) + e)
    a, _, ea, _ = act(L, kind, z)
    ey = (e if kind in (L.QB_ACT_NONE, L.QB_ACT_RELU) else 1.13 * e + e * e) + ea
    if residual is not None:
        a = a + residual
        ey = ey + U * (np.abs(a) + ey)
    return z, e, a, ey


def gated(L, x, wg, wu, kind):
    """(g, its error, u, its error, y, its error)."""
    g, eg = product(x, wg)
    u, eu = product(x, wu)
    a, _, ea, _ = act(L, kind, g)
    ea = ea + 1.13 * eg + eg * eg
    y = a * u
    return g, eg, u, eu, y, ea * np.abs(u) + eu * np.abs(a) + ea * eu + U * np.abs(y)


def rounded_product(dz, e_dz, w, dt):
    """dz w for a dz that is off by e_dz and then rounded to dt, and its error."""
    n = dz.shape[1]
    total = np.abs(dz) + e_dz
    err = e_dz @ np.abs(w) + (n + 2) * 2 * U * (total @ np.abs(w))
    if dt != torch.float32:
        h = half_step(dt, total)
        err = err + np.minimum(h @ np.abs(w), 7 * np.sqrt((h * h) @ (w * w)))
    return dz @ w, err
