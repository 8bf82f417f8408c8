"""GPU: arrays and weights beyond 2^32 elements or bytes in the 4-bit layers, their gradients and the
gradient norm: sampled rows and columns against the binary64 formulas (linear_reference.py)."""
import math

import numpy as np
import pytest
import torch

import linear_reference as ref
import oracle
import test_gpu_gated as gated
import test_gpu_grad_norm as clip
import test_gpu_linear as linear
from gpu_helpers import DEV, qb

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def spread(count, size):
    return sorted({0, 1, size - 1, size - 2, *(i * (size // count) + i for i in range(count))})


@pytest.mark.parametrize("K", [32, 64])
def test_activations_beyond_32_bits(K):
    """131075 rows of 16500 outputs (2.16e9 elements), by the rows kernel (K = 32) and by the tiled product."""
    L = qb()
    M, N = 131075, 16500
    w = gated.pair(N, K, oracle.NF4, 64, False, BF16, 1)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    x = torch.empty(M, K, dtype=BF16, device=DEV).normal_(generator=gen)
    bias = ref.normal((N,), 2)
    at = torch.tensor(spread(12, M), device=DEV)
    y, z = linear.forward(L, x, w[0], bias, "SILU", keep=True)
    linear.check_forward(L, x[at], w[0], bias, "SILU", None, y[at], z[at])
    dy = torch.empty(M, N, dtype=BF16, device=DEV).normal_(0, 0.1, generator=gen)
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


class Rows:
    """Some rows (or columns) of a weight whose values are on the host."""

    def __init__(self, values):
        self.values, self.w = values, values.double().numpy()


@pytest.mark.parametrize("M", [2, 70])
def test_weight_beyond_32_bits(M):
    """A weight of 2^20 + 5 by 8192 (8.6e9 elements, 4.3 GB of codes): outputs from all over it, and the input's gradient
    for a dy that is zero but for a few outputs."""
    L = qb()
    N, K = (1 << 20) + 5, 8192
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    codes = torch.randint(0, 256, (N * K // 2,), dtype=torch.uint8, device=DEV, generator=gen)
    absmax = torch.rand(N * K // 64, device=DEV, generator=gen) * 0.1 + 0.005
    at = spread(10, N)
    rows = []
    for n in at:
        c = codes[n * K // 2:(n + 1) * K // 2].cpu().numpy()
        a = absmax[n * K // 64:(n + 1) * K // 64].cpu().numpy()
        rows.append(oracle.dequantize_blockwise(c, a, oracle.NF4, 64, K, ydt=ref.DT_OF[BF16]).view(np.int16))
    some = Rows(torch.from_numpy(np.stack(rows)).view(BF16))
    at = torch.tensor(at, device=DEV)
    x = ref.normal((M, K), 1, dtype=BF16)
    ws = torch.empty(L.qb_dequant_linear_workspace_bytes(L.QB_BF16, M, K, N) + 16, dtype=torch.uint8, device=DEV)
    y = torch.empty(M, N, dtype=BF16, device=DEV)
    L.qb_dequant_linear(x, codes, absmax, oracle.NF4, 64, N, y, ws)
    torch.cuda.synchronize()
    linear.check_forward(L, x, some, None, "NONE", None, y[:, at].contiguous())
    del ws
    torch.cuda.empty_cache()
    dy = torch.zeros(M, N, dtype=BF16, device=DEV)
    part = ref.normal((M, len(at)), 2, dtype=BF16)
    dy[:, at] = part
    ws = torch.empty(L.qb_dequant_linear_backward_workspace_bytes(L.QB_BF16, M, K, N), dtype=torch.uint8, device=DEV)
    dx = torch.empty(M, K, dtype=BF16, device=DEV)
    L.qb_dequant_linear_backward(dy, codes, absmax, oracle.NF4, 64, K, dx, ws)
    torch.cuda.synchronize()
    linear.check_backward(L, part, some, None, "NONE", dx, None, None)


def test_gradient_beyond_32_bits():
    """2^32 + 70001 elements in bf16 beside a short gradient: all ones but for one near the end."""
    L = qb()
    n = (1 << 32) + 70001
    g = torch.ones(n, dtype=BF16, device=DEV)
    g[n - 3] = 65536.0
    short = torch.full((5,), 2.0, device=DEV)
    table = L.grad_table([g, short])
    norm = torch.empty(1, device=DEV)
    ws = torch.empty(L.qb_multi_tensor_grad_norm_workspace_bytes(2), dtype=torch.uint8, device=DEV)
    L.qb_multi_tensor_grad_norm(table, 2, norm, ws)
    want = math.sqrt(n - 1 + 2.0 ** 32 + 20)
    assert abs(norm.item() - want) <= want * 2.0 ** -24 * 1.001
    L.qb_multi_tensor_clip_grads(table, 2, want / 4, norm)
    torch.cuda.synchronize()
    # the scale is within 2^-23 of 1 / 4 (the norm is rounded to binary32), which bf16 does not show
    ones = bool((g[:n - 3] == 0.25).all()) and bool((g[n - 2:] == 0.25).all())
    assert ones and g[n - 3].item() == 16384.0
    assert torch.equal(short, clip.expected(torch.full_like(short, 2.0), want / 4, norm))
