"""GPU: statistics of rows whose spread is small against their mean, for every
type and every way that a row is spread over threads.

Rows of equal values x.  The first mean m0 is off by delta, at most (L + 2) u |x|; the
differences x - m0 are exact (x and m0 within a factor of two), multiples of the
last place of x by a small whole number, so their sum is exact and its mean c is
off by 2 u delta at most: m0 + c rounds to x.  So the mean is x, every normalized
value is zero, and with them the weight's gradient."""
import numpy as np
import pytest
import torch

import layers_reference as ref
from gpu_helpers import DEV, qb

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]
EPS = 1e-5
# numbers of elements that are no powers of two, whole and ragged, for every way of spreading a row over
# threads (an ordinary width of 896 among them), and two beyond the registers
DIMS = [3, 65, 127, 159, 500, 896, 1126, 1500, 2050, 3600, 4099, 5199, 9000, 16000, 16387, 20000]
VALUES = [3.0, -1000.0, 60000.0, 0.0, 1.0 / 3.0, -4096.0]


def constant_rows(values, dim, dt):
    return torch.tensor(values, device=DEV).to(dt)[:, None].expand(len(values), dim).contiguous()


def norm(L, x):
    y = torch.full_like(x, 7.0)
    mean, rstd = (torch.full((x.shape[0],), 7.0, device=DEV) for _ in range(2))
    L.qb_layer_norm(x, None, None, EPS, y, mean=mean, rstd=rstd)
    return y, mean, rstd


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("dim", DIMS)
def test_rows_of_equal_values(dim, dt):
    L = qb()
    x = constant_rows(VALUES, dim, dt)
    y, mean, rstd = norm(L, x)
    assert torch.equal(mean, x[:, 0].float())
    assert (y == 0).all()
    # The squared differences n delta^2 are taken off again up to (L + 6) u of them; rstd is off by half of
    # what is left against eps, and by 3 u of its own.
    delta = (ref.L + 2) * ref.U * np.abs(ref.f64(x[:, 0]))
    left = delta ** 2 * (ref.L + 6) * ref.U / EPS
    want = 1 / np.sqrt(np.full(len(VALUES), float(np.float32(EPS))))
    ref.assert_close(rstd, want, want * (left / 2 + 3 * ref.U), "rstd")


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("dim", DIMS)
def test_means_far_from_zero(dim, dt):
    """The bounds of binary32 rows (mean: its own rounding and 50 u of the spread) hold for 16-bit rows too."""
    L = qb()
    g = torch.Generator(device=DEV)
    g.manual_seed(dim)
    x = (1000 + 8 * torch.randint(-3, 4, (40, dim), device=DEV, generator=g).float()).to(dt)
    x[20:] = (30000 + 256 * torch.randint(0, 2, (20, dim), device=DEV, generator=g).float()).to(dt)
    y, mean, rstd = norm(L, x)
    want, err, m, r, e_m, e_r = ref.layer_norm(ref.f64(x), None, None, float(np.float32(EPS)), True)
    ref.assert_close(y, want, err, "y")
    ref.assert_close(mean, m, e_m, "mean")
    ref.assert_close(rstd, r, e_r, "rstd")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("n", [50, 300])
def test_stable_embedding_of_equal_values(n, dt):
    """A lookup scaled by 0.7 has binary32 values whatever the table's type; both forms of the gradient."""
    L = qb()
    rows = len(VALUES)
    for dim in [d for d in DIMS if d <= 16384]:
        table = constant_rows(VALUES, dim, dt)
        ids = torch.arange(n, device=DEV) % rows
        y = torch.full((n, dim), 7.0, device=DEV)
        L.qb_stable_embedding(table, ids, None, None, EPS, y, scale=0.7)
        assert (y == 0).all(), dim
        dy = torch.empty(n, dim, device=DEV).normal_(0, 1)
        ws = torch.empty(L.qb_stable_embedding_workspace_bytes(n, rows, dim), dtype=torch.uint8, device=DEV)
        dtable = torch.empty(rows, dim, device=DEV)
        dgamma = torch.full((dim,), 7.0, device=DEV)
        L.qb_stable_embedding_backward(dy, table, ids, None, EPS, dtable, dgamma, None, ws, scale=0.7)
        assert (dgamma == 0).all(), dim


# Rows whose squared differences from a rounded mean are almost all the mean's own rounding, or overflow binary32.
LARGE = [1e8 / 3, -1e12, 1e19 / 7, 3e25, -1e30, 1e33 / 3]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("dim", DIMS)
def test_large_rows_of_equal_values(dim, dt):
    """The variance is zero whatever the value is: the differences from m0 + c, rounded to one binary32, are
    exactly zero."""
    L = qb()
    x = constant_rows(LARGE, dim, dt)
    y, mean, rstd = norm(L, x)
    assert torch.equal(mean, x[:, 0].float())
    assert (y == 0).all()
    want = 1 / np.sqrt(np.full(len(LARGE), float(np.float32(EPS))))
    ref.assert_close(rstd, want, want * 3 * ref.U, "rstd")
    if dim > 16384:
        return
    # the same statistics inside the stable embedding and its gradient: h = 0, dtable = rstd (dy - mean dy)
    ids = torch.arange(len(LARGE), device=DEV)
    z = torch.full_like(x, 7.0)
    L.qb_stable_embedding(x, ids, None, None, EPS, z)
    assert (z == 0).all()
    dy = torch.empty(len(LARGE), dim, device=DEV).normal_(0, 1)
    ws = torch.empty(L.qb_stable_embedding_workspace_bytes(len(LARGE), len(LARGE), dim), dtype=torch.uint8, device=DEV)
    dtable, dgamma = torch.empty_like(dy), torch.full((dim,), 7.0, device=DEV)
    L.qb_stable_embedding_backward(dy, x, ids, None, EPS, dtable, dgamma, None, ws)
    assert (dgamma == 0).all()
    d = ref.f64(dy)
    err_r = want * 3 * ref.U
    g, err = ref.norm_grad(d, np.zeros_like(d), np.zeros_like(d), np.zeros_like(d), want, err_r, np.ones(dim))
    ref.assert_close(dtable, g, err, "dtable")


@pytest.mark.parametrize("dim", DIMS)
def test_spreads_of_the_last_place(dim):
    """x = a + k s with whole k and s the last place of a: differences from any mean that is a multiple of s
    are exact, so the variance keeps its digits."""
    L = qb()
    g = torch.Generator(device=DEV)
    g.manual_seed(dim)
    k = torch.randint(-3, 4, (40, dim), device=DEV, generator=g).float()
    k[::4] = (k[::4] == 3).float()
    a = torch.tensor([1e6, 1e4, -3e8, 5e10], device=DEV).repeat(10)[:, None]
    s = 2.0 ** torch.floor(torch.log2(a.abs()) - 23)
    x = (a + k * s).contiguous()
    assert torch.equal((x - a) / s, k)
    y, mean, rstd = norm(L, x)
    xd = ref.f64(x)
    m, _, r = ref.statistics(xd, float(np.float32(EPS)))
    # the mean: its own rounding and the correction's.  rstd: at most half of the squared differences are the
    # mean's, so what is left of them is off by 2 (L + 6) u.
    ref.assert_close(mean, m, ref.U * np.abs(m) + (ref.L + 2) * ref.U / r, "mean")
    ref.assert_close(rstd, r, r * ((2 * (ref.L + 6)) / 2 + 3) * ref.U, "rstd")


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("dim", [d for d in DIMS if d > 3])
def test_variance_beyond_binary32(dim, dt):
    """Differences whose squares overflow: var is infinite, 1 / sqrt(var + eps) zero, and y is beta."""
    L = qb()
    g = torch.Generator(device=DEV)
    g.manual_seed(dim)
    x = (1e25 * (torch.randn(8, dim, device=DEV, generator=g) + 3 * torch.randn(8, 1, device=DEV, generator=g))).to(dt)
    y, mean, rstd = norm(L, x)
    assert (y == 0).all() and (rstd == 0).all()
    xd = ref.f64(x)
    ref.assert_close(mean, xd.mean(1), ref.U * np.abs(xd.mean(1)) + (ref.L + 2) * ref.U * xd.std(1), "mean")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("dim", DIMS + [64, 1024, 2048, 8192])
def test_means_of_rows_that_hold_infinities(dim, dt):
    """The mean is the infinity (NaN for both of them), as sum x / dim; var, rstd and y are NaN, inf - inf."""
    L = qb()
    inf, nan = float("inf"), float("nan")
    g = torch.Generator(device=DEV)
    g.manual_seed(dim)
    x = torch.randn(9, dim, device=DEV, generator=g)
    x[1, 0] = inf
    x[2, dim - 1] = -inf
    x[3, dim // 2] = inf
    x[3, dim // 3] = inf
    x[4, 0], x[4, dim - 1] = inf, -inf
    x[5, dim // 2] = nan
    x[6] = inf
    x[7, 0], x[7, dim // 2] = inf, nan
    want = torch.tensor([inf, -inf, inf, nan, nan, inf, nan], device=DEV)
    x = x.to(dt)
    clean = norm(L, x[::8].clone())
    y, mean, rstd = norm(L, x)
    assert torch.equal(mean[1:8].nan_to_num(nan=5.0), want.nan_to_num(nan=5.0))
    assert rstd[1:8].isnan().all() and y[1:8].isnan().all()
    for got, alone in zip((y, mean, rstd), clean):
        assert torch.equal(got[::8], alone)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("dim", DIMS + [64, 4096])
def test_gradients_of_very_large_rows_of_equal_values(dim, dt):
    """|mean| * rstd overflows, which only an element outside the row would meet: h = 0 in the row, so
    dx = rstd (g - mean g), dgamma = 0."""
    L = qb()
    x = constant_rows([1e34, -3e33, 2.0, 1e33] * 10, dim, dt)[:37 if dim < 5000 else 5]
    n, eps = x.shape[0], 1e-12
    y = torch.full_like(x, 7.0)
    mean, rstd = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    L.qb_layer_norm(x, None, None, eps, y, mean=mean, rstd=rstd)
    assert (y == 0).all() and torch.equal(mean, x[:, 0].float())
    r = ref.f64(rstd)
    dy = torch.empty(n, dim, device=DEV).normal_(0, 1).to(dt)
    dx = torch.full_like(x, 7.0)
    dgamma = torch.full((dim,), 7.0, device=DEV)
    ws = torch.empty(L.qb_layer_norm_workspace_bytes(n, dim), dtype=torch.uint8, device=DEV)
    L.qb_layer_norm_backward(dy, x, None, mean, rstd, dx, dgamma, None, ws)
    d = ref.f64(dy)
    zero = np.zeros_like(d)
    want, err = ref.norm_grad(d, zero, zero, zero, r, np.zeros_like(r), np.ones(dim))
    ref.assert_close(dx, want, err, "dx")
    assert (dgamma == 0).all()
    if dim > 16384:
        return
    for m in (n, 200):                                  # both forms of the table's gradient
        ids = torch.arange(m, device=DEV) % n
        dy = torch.empty(m, dim, device=DEV).normal_(0, 1)
        dtable = torch.full((n, dim), 7.0, device=DEV)
        ws = torch.empty(L.qb_stable_embedding_workspace_bytes(m, n, dim), dtype=torch.uint8, device=DEV)
        L.qb_stable_embedding_backward(dy, x, ids, None, eps, dtable, dgamma, None, ws)
        s, e_s, _ = ref.token_sums(ref.f64(dy), ids.tolist(), n)
        want, err = ref.norm_grad(s, e_s, np.zeros_like(s), np.zeros_like(s), r, 3 * ref.U * r, np.ones(dim))
        ref.assert_close(dtable, want, err, f"dtable of {m} tokens")
        assert (dgamma == 0).all()
