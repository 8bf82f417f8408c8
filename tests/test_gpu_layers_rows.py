"""GPU: a row's result does not depend on the rows beside it.  A workgroup takes
many rows in turn; each must come out with the bits that it has in a call of
a few rows, where every workgroup takes one (statistics of neighbouring rows, which
differ by orders of magnitude here, never mix)."""
import pytest
import torch

from gpu_helpers import DEV, qb

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
DIMS = [64, 500, 1024, 2048, 2049, 4096, 5003, 8192, 16384]


def rows(n, dim, dt, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(n, dim, device=DEV, generator=g)
    size = torch.pow(10.0, torch.randint(-3, 3, (n, 1), device=DEV, generator=g).float())
    return ((x + torch.randn(n, 1, device=DEV, generator=g)) * size).to(dt)


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("dim", DIMS)
def test_layer_norm(dim, dt):
    L = qb()
    n = 6000
    x = rows(n, dim, dt, dim)
    w = torch.randn(dim, device=DEV), torch.randn(dim, device=DEV)
    y, few = torch.empty_like(x), torch.empty_like(x)
    stats, some = torch.empty(2, n, device=DEV), torch.empty(2, n, device=DEV)
    L.qb_layer_norm(x, w[0], w[1], 1e-5, y, mean=stats[0], rstd=stats[1])
    for t in range(0, n, 256):
        m = min(256, n - t)
        a, b = torch.empty(m, device=DEV), torch.empty(m, device=DEV)
        out = torch.empty(m, dim, dtype=dt, device=DEV)
        L.qb_layer_norm(x[t:t + m].clone(), w[0], w[1], 1e-5, out, mean=a, rstd=b)
        few[t:t + m], some[0, t:t + m], some[1, t:t + m] = out, a, b
    assert torch.equal(stats, some)
    assert torch.equal(y, few)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("dim", DIMS)
def test_stable_embedding(dim, dt):
    """... also with ids outside the table between the others."""
    L = qb()
    n, count = 6000, 900
    table = rows(count, dim, dt, dim + 1)
    g = torch.Generator(device=DEV)
    g.manual_seed(dim)
    ids = torch.randint(-300, count, (n,), device=DEV, generator=g)
    w = torch.randn(dim, device=DEV), torch.randn(dim, device=DEV)
    y = torch.empty(n, dim, dtype=dt, device=DEV)
    L.qb_stable_embedding(table, ids, w[0], w[1], 1e-5, y, scale=1.5)
    for t in range(0, n, 256):
        m = min(256, n - t)
        out = torch.empty(m, dim, dtype=dt, device=DEV)
        L.qb_stable_embedding(table, ids[t:t + m].clone(), w[0], w[1], 1e-5, out, scale=1.5)
        assert torch.equal(y[t:t + m], out)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("dim", DIMS)
def test_layer_norm_backward(dim, dt):
    L = qb()
    n = 6000
    x, dy = rows(n, dim, dt, dim + 2), rows(n, dim, dt, dim + 3)
    gamma = torch.randn(dim, device=DEV)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    L.qb_layer_norm(x, gamma, None, 1e-5, y, mean=mean, rstd=rstd)
    L.qb_layer_norm_backward(dy, x, gamma, mean, rstd, dx, None, None)
    for t in range(0, n, 256):
        m = min(256, n - t)
        out = torch.empty(m, dim, dtype=dt, device=DEV)
        L.qb_layer_norm_backward(dy[t:t + m].clone(), x[t:t + m].clone(), gamma, mean[t:t + m].clone(),
                                 rstd[t:t + m].clone(), out, None, None)
        assert torch.equal(dx[t:t + m], out)
