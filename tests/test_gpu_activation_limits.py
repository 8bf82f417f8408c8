"""GPU: activations and their derivatives at infinite and NaN pre-activations: the limits at the infinities
(0 and 0 at the negative one, infinity and 1 at the positive one), and NaN at NaN, in every kernel that takes
them; a gate that fp16 cannot hold leaves its row's gradient finite."""
import pytest
import torch

import linear_reference as ref
import oracle
import test_gpu_gated as gated
import test_gpu_linear as linear
from gpu_helpers import DEV, qb

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NAN, INF = float("nan"), float("inf")
ACTS = ["RELU", "GELU", "GELU_TANH", "SILU"]


def special(n, xdt=F32):
    """Ordinary values, and at three places of every twelve infinity, its negative and NaN."""
    z = ref.normal((n,), 5, 2.0, xdt)
    z[1::12], z[5::12], z[8::12] = INF, -INF, NAN
    return z


def limits(z, act):
    """act(z) and act'(z) at the places that are not finite."""
    value = torch.where(z == -INF, torch.zeros_like(z), z)
    slope = torch.where(z == INF, torch.ones_like(z), torch.where(z == -INF, torch.zeros_like(z), z))
    return value, slope


def same(a, b):
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(7.0, INF, -INF), b.nan_to_num(7.0, INF, -INF))


@pytest.mark.parametrize("M", [3, 20, 60, 1100])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("xdt", [BF16, F16, F32])
def test_linear_layer(M, act, xdt):
    """Infinite and NaN biases under products of zero; columns in whole groups and beyond them."""
    L = qb()
    N, K = 85, 160
    w = ref.Weight(N, K, oracle.NF4, 64, False, xdt, seed=1)
    bias = special(N)
    odd = ~bias.isfinite()
    value, slope = limits(bias.to(xdt), act)
    x = torch.zeros(M, K, dtype=xdt, device=DEV)
    y, z = linear.forward(L, x, w, bias, act, keep=True)
    assert same(z, bias.to(xdt).expand(M, N))
    assert same(y[:, odd], value[odd].expand(M, -1)), y[0, odd]
    assert y[:, ~odd].isfinite().all()
    dy = torch.ones(M, N, dtype=xdt, device=DEV)
    dz = linear.backward(L, dy, w, z, act, dx=False, dz=True)[1]
    assert same(dz[:, odd], slope[odd].expand(M, -1)), dz[0, odd]
    assert dz[:, ~odd].isfinite().all()
    # NaN reaches its row's dx, the infinities leave it as the limits do
    z[1:] = torch.where(z[1:].isnan(), torch.zeros_like(z[1:]), z[1:])
    dx = linear.backward(L, dy, w, z, act)[0]
    assert dx[0].isnan().all() and dx[1:].isfinite().all()


@pytest.mark.parametrize("M", [3, 60, 1100])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("xdt", [BF16, F16, F32])
def test_gated_gradients(M, act, xdt):
    L = qb()
    N, K = 85, 160
    w = gated.pair(N, K, oracle.NF4, 64, False, xdt, 1)
    g = special(N, xdt).expand(M, N).contiguous()
    odd = ~g[0].isfinite()
    value, slope = limits(g[0], act)
    dy, u = torch.ones(M, N, dtype=xdt, device=DEV), torch.full((M, N), 2.0, dtype=xdt, device=DEV)
    _, dg, du = gated.backward(L, dy, g, u, w, act, dx=False, keep=(True, True))
    assert same(dg[:, odd], 2.0 * slope[odd].expand(M, -1)), dg[0, odd]
    assert same(du[:, odd], value[odd].expand(M, -1)), du[0, odd]
    assert dg[:, ~odd].isfinite().all() and du[:, ~odd].isfinite().all()


@pytest.mark.parametrize("M", [3, 60, 1100])
@pytest.mark.parametrize("act", ACTS)
def test_gate_beyond_fp16(M, act):
    """Sums below -65504 are kept as -inf in fp16: y and every gradient are finite."""
    L = qb()
    N, K = 40, 160
    w = gated.pair(N, K, oracle.NF4, 64, False, F16, 1)
    w[0].codes.fill_(0x00)                               # all -1 times a positive constant
    x = torch.full((M, K), 2000.0, dtype=F16, device=DEV)
    w[0].absmax.fill_(0.5)
    y, g, u = gated.forward(L, x, w, act, keep=True)
    assert (g == -INF).all() and u.isfinite().all() and (y == 0).all()
    dy = ref.normal((M, N), 3, 1.0, F16)
    dx, dg, du = gated.backward(L, dy, g, u, w, act, keep=(True, True))
    assert (dg == 0).all() and (du == 0).all() and (dx == 0).all()
