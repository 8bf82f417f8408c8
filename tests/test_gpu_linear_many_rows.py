"""GPU: calls of the 4-bit layers that are cut into several launches of fewer rows each, and activations beyond
2^32 elements: sampled rows and columns against the binary64 formulas (linear_reference.py)."""
import numpy as np
import pytest
import torch

import linear_reference as ref
import oracle
import test_gpu_gated as gated
import test_gpu_linear as linear
from gpu_helpers import DEV, qb
from test_gpu_linear import BF16, F32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def random(shape, seed, std=1.0, xdt=BF16):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.empty(shape, dtype=xdt, device=DEV).normal_(0, std, generator=g)


def around(cut, size):
    """Both ends, the rows around a cut, and some between."""
    rows = {*range(4), *range(cut - 70, cut + 70), *range(size - 70, size), *(i * (size // 200) + i for i in range(200))}
    return torch.tensor(sorted(r for r in rows if 0 <= r < size), device=DEV)


@pytest.mark.parametrize("xdt,cut", [(BF16, 1 << 21), (F32, 1 << 20)])
def test_rows_kernel_in_two_launches(xdt, cut):
    """32 inputs: the rows kernel takes any number of rows, 32768 workgroups of them a launch."""
    L = qb()
    M, K, N = cut + 70, 32, 17
    w = gated.pair(N, K, oracle.NF4, 64, False, xdt, 1)
    x, residual, bias = random((M, K), 1, 1.0, xdt), random((M, N), 2, 1.0, xdt), ref.normal((N,), 3)
    at = around(cut, M)
    y, z = linear.forward(L, x, w[0], bias, "SILU", residual, keep=True)
    linear.check_forward(L, x[at], w[0], bias, "SILU", residual[at], y[at], z[at])
    assert torch.equal(linear.forward(L, x, w[0], bias, "SILU", residual, in_place=True), y)
    y, g, u = gated.forward(L, x, w, "GELU", keep=True)
    gated.check_forward(L, x[at], w, "GELU", y[at], g[at], u[at])
    assert all(t.isfinite().all() for t in (y, g, u, z))


class Columns:
    """Some outputs of a weight."""

    def __init__(self, w, at):
        self.w = w.w[at]


def test_tiled_product_in_two_calls():
    """2^21 - 1 outputs: 16384 rows at a time (a gated block 8192); bias with every piece."""
    L = qb()
    K, N = 64, (1 << 21) - 1
    w = gated.pair(N, K, oracle.NF4, 64, False, BF16, 1)
    cols = sorted({0, 1, 15, 16, N - 1, N - 2, N - 17, *(i * (N // 40) + i for i in range(40))})
    some, at_cols = [Columns(v, cols) for v in w], torch.tensor(cols, device=DEV)
    M, cut = 16384 + 70, 16384
    x, bias, at = random((M, K), 1), ref.normal((N,), 2), around(16384, 16384 + 70)
    y = linear.forward(L, x, w[0], bias, "SILU")
    linear.check_forward(L, x[at], some[0], bias[at_cols], "SILU", None, y[at][:, at_cols])
    assert y[cut - 1:].isfinite().all()
    del y
    torch.cuda.empty_cache()
    M, cut = 8192 + 70, 8192
    at = around(cut, M)
    y = gated.forward(L, x[:M], w, "SILU")
    want_g, eg, want_u, eu, want, e = ref.gated(L, ref.f64(x[at]), some[0].w, some[1].w, L.QB_ACT_SILU)
    ref.assert_close(y[at][:, at_cols], want, e, "y")
    assert y[cut - 1:].isfinite().all()


def test_input_gradient_in_two_calls():
    """2^21 - 32 inputs: dx 16384 rows at a time, the bias's gradient once, over all rows."""
    L = qb()
    K, N, cut = (1 << 21) - 32, 64, 16384
    M = cut + 70
    w = ref.Weight(N, K, oracle.NF4, 64, True, BF16, seed=1)
    dy = random((M, N), 1)
    dx, _, db = linear.backward(L, dy, w, bias_dt=F32)
    at = around(cut, M)
    cols = sorted({0, 1, 31, 32, K - 1, K - 33, *(i * (K // 40) + i for i in range(40))})
    d = ref.f64(dy[at])
    got = dx[at][:, torch.tensor(cols, device=DEV)]
    ref.assert_close(got, *ref.rounded_product(d, np.zeros_like(d), w.w[:, cols], BF16), "dx")
    linear.check_backward(L, dy, w, None, "NONE", None, None, db)
    assert dx[cut - 1:].isfinite().all()


@pytest.mark.parametrize("K", [32, 64])
def test_more_than_2_to_the_32_elements(K):
    """262150 rows of 16500 outputs (4.3e9 elements), by the rows kernel (32 inputs) and by the tiled product, with
    their gradients."""
    L = qb()
    M, N = 262150, 16500
    assert M * N > 1 << 32
    w = gated.pair(N, K, oracle.NF4, 64, False, BF16, 1)
    x, bias = random((M, K), 1), ref.normal((N,), 2)
    at = torch.tensor(sorted({0, 1, M - 1, M - 2, *(i * (M // 12) + i for i in range(12))}), device=DEV)
    y, z = linear.forward(L, x, w[0], bias, "SILU", keep=True)
    linear.check_forward(L, x[at], w[0], bias, "SILU", None, y[at], z[at])
    del y
    dy = random((M, N), 3, 0.1)
    dx, dz, _ = linear.backward(L, dy, w[0], z, "SILU", dz=True)
    linear.check_backward(L, dy[at], w[0], z[at], "SILU", dx[at], dz[at], None)
    assert dx.isfinite().all()
    del z, dz, dx
    torch.cuda.empty_cache()
    y, g, u = gated.forward(L, x, w, keep=True)
    gated.check_forward(L, x[at], w, "SILU", y[at], g[at], u[at])
    del y
    dx = gated.backward(L, dy, g, u, w)[0]
    gated.check_backward(L, dy[at], g[at], u[at], w, "SILU", dx[at])
    assert dx.isfinite().all()
