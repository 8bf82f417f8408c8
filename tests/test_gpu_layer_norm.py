"""GPU: layer norm and its backward pass against the binary64 formulas, within
the rounding error of a binary32 evaluation (layers_reference.py)."""
import numpy as np
import pytest
import torch

import layers_reference as ref
from gpu_helpers import DEV, qb

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-5
PAIRS = [(F32, F32), (F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)]
# every way a row is spread over threads, whole and ragged, and rows beyond the registers
DIMS = [1, 3, 8, 100, 128, 129, 512, 600, 1024, 1500, 2048, 2049, 4096, 5001, 8192, 9000, 16384, 16387, 40000]


def data(n, dim, xdt, wdt, seed, offset=0.5):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.empty(n, dim, device=DEV).normal_(0, 1, generator=g)
    x = (x * (0.5 + torch.rand(dim, device=DEV, generator=g)) + offset * torch.randn(n, 1, device=DEV, generator=g)).to(xdt)
    gamma = (1 + 0.2 * torch.randn(dim, device=DEV, generator=g)).to(wdt)
    beta = (0.2 * torch.randn(dim, device=DEV, generator=g)).to(wdt)
    dy = (0.1 * torch.randn(n, dim, device=DEV, generator=g)).to(xdt)
    return x, gamma, beta, dy


def forward(L, x, gamma, beta, eps=EPS):
    n = x.shape[0]
    y = torch.full((n + 1, x.shape[1]), 7.0, dtype=x.dtype, device=DEV)
    mean, rstd = torch.full((n,), 7.0, device=DEV), torch.full((n,), 7.0, device=DEV)
    L.qb_layer_norm(x, gamma, beta, eps, y[:n], mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    assert (y[n:] == 7.0).all()                        # nothing behind the last row
    return y[:n], mean, rstd


def check_forward(x, gamma, beta, y, mean, rstd, eps=EPS):
    want, err, m, r, e_m, e_r = ref.layer_norm(ref.f64(x), None if gamma is None else ref.f64(gamma),
                                               None if beta is None else ref.f64(beta), float(np.float32(eps)),
                                               x.dtype == F32 or x.shape[1] > 16384)
    ref.assert_close(y, want, err, "y")
    ref.assert_close(mean, m, e_m, "mean")
    ref.assert_close(rstd, r, e_r, "rstd")


def check_backward(x, gamma, dy, mean, rstd, dx, dgamma, dbeta, old=None):
    """The statistics are inputs: h is off by the difference's and the product's roundings only."""
    xd, m, r = ref.f64(x), ref.f64(mean), ref.f64(rstd)
    h = (xd - m[:, None]) * r[:, None]
    e_h = 2 * ref.U * np.abs(h)
    d = ref.f64(dy)
    g = np.ones(x.shape[1]) if gamma is None else ref.f64(gamma)
    if dx is not None:
        want, err = ref.norm_grad(d, np.zeros_like(d), h, e_h, r, np.zeros_like(r), g)
        ref.assert_close(dx, want, err, "dx")
    for got, terms, e in ((dgamma, d * h, np.abs(d) * e_h), (dbeta, d, np.zeros_like(d))):
        if got is None:
            continue
        want, err = ref.column_sum(terms, e)
        if old is not None:
            want = want + ref.f64(old)
            err = err + ref.U * np.abs(want)
        ref.assert_close(got, want, err, "dgamma, dbeta")


def backward(L, x, gamma, dy, mean, rstd, wdt):
    n, dim = x.shape
    ws = torch.full((L.qb_layer_norm_workspace_bytes(n, dim),), 0xCD, dtype=torch.uint8, device=DEV)
    buf = torch.full((n + 1, dim), 7.0, dtype=x.dtype, device=DEV)
    dg, db = (torch.full((dim + 8,), 7.0, dtype=wdt, device=DEV) for _ in range(2))
    L.qb_layer_norm_backward(dy, x, gamma, mean, rstd, buf[:n], dg[:dim], db[:dim], ws)
    torch.cuda.synchronize()
    assert (buf[n:] == 7.0).all() and (dg[dim:] == 7.0).all() and (db[dim:] == 7.0).all()
    return buf[:n], dg[:dim], db[:dim]


@pytest.mark.parametrize("xdt,wdt", PAIRS)
@pytest.mark.parametrize("dim", DIMS)
def test_forward_and_backward(xdt, wdt, dim):
    L = qb()
    for n in (1, 2, 37) if dim < 10000 else (1, 5):
        x, gamma, beta, dy = data(n, dim, xdt, wdt, dim + n)
        y, mean, rstd = forward(L, x, gamma, beta)
        check_forward(x, gamma, beta, y, mean, rstd)
        dx, dg, db = backward(L, x, gamma, dy, mean, rstd, wdt)
        check_backward(x, gamma, dy, mean, rstd, dx, dg, db)


@pytest.mark.parametrize("n,dim,xdt", [(3001, 64, BF16), (2777, 300, F32), (5000, 16, F16), (1300, 2048, BF16), (1029, 4100, F32)])
def test_many_rows(n, dim, xdt):
    """Several rows per thread and workgroup; the same bits on a second run."""
    L = qb()
    x, gamma, beta, dy = data(n, dim, xdt, F32, n)
    y, mean, rstd = forward(L, x, gamma, beta)
    check_forward(x, gamma, beta, y, mean, rstd)
    first = backward(L, x, gamma, dy, mean, rstd, F32)
    check_backward(x, gamma, dy, mean, rstd, *first)
    again = backward(L, x, gamma, dy, mean, rstd, F32)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("dim", [96, 1003, 20000])
def test_optional_arguments(dim):
    """gamma, beta, the statistics and each gradient may be left out."""
    L = qb()
    n = 19
    x, gamma, beta, dy = data(n, dim, BF16, BF16, dim)
    for g, b in ((None, None), (gamma, None), (None, beta)):
        y, mean, rstd = forward(L, x, g, b)
        check_forward(x, g, b, y, mean, rstd)
    y2 = torch.empty_like(x)
    L.qb_layer_norm(x, None, beta, EPS, y2)
    assert torch.equal(y, y2)
    ws = torch.empty(L.qb_layer_norm_workspace_bytes(n, dim), dtype=torch.uint8, device=DEV)
    full = backward(L, x, None, dy, mean, rstd, BF16)
    check_backward(x, None, dy, mean, rstd, *full)
    for keep in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 1, 1)):
        out = [torch.empty_like(t) if k else None for t, k in zip(full, keep)]
        L.qb_layer_norm_backward(dy, x, None, mean, rstd, *out, ws if keep[1] or keep[2] else None)
        assert all(o is None or torch.equal(o, t) for o, t in zip(out, full))


@pytest.mark.parametrize("wdt", [F32, BF16])
def test_weight_gradients_accumulate(wdt):
    L = qb()
    n, dim = 200, 777
    x, gamma, beta, dy = data(n, dim, BF16, wdt, 3)
    _, mean, rstd = forward(L, x, gamma, beta)
    ws = torch.empty(L.qb_layer_norm_workspace_bytes(n, dim), dtype=torch.uint8, device=DEV)
    old = torch.randn(dim, device=DEV).to(wdt)
    dx, dg, db = torch.full_like(x, 7.0), old.clone(), old.clone()
    L.qb_layer_norm_backward(dy, x, gamma, mean, rstd, dx, dg, db, ws, accumulate=True)
    check_backward(x, gamma, dy, mean, rstd, dx, dg, db, old=old)
    # no rows: left as they are with accumulate, zero without
    none = torch.empty(0, dim, dtype=BF16, device=DEV)
    stat = torch.empty(0, device=DEV)
    L.qb_layer_norm_backward(none, none, gamma, stat, stat, none, dg, db, ws, accumulate=True)
    check_backward(x, gamma, dy, mean, rstd, dx, dg, db, old=old)
    L.qb_layer_norm_backward(none, none, gamma, stat, stat, none, dg, db, ws)
    assert (dg == 0).all() and (db == 0).all()
    L.qb_layer_norm(none, gamma, beta, EPS, none)


def test_rows_of_equal_values_and_far_means():
    """A constant row has h = 0 up to the mean's rounding; a mean that is large
    against the spread keeps its digits."""
    L = qb()
    for dim in (100, 1001, 2500, 4096, 7000, 16383, 16385):
        g = torch.Generator(device=DEV)
        g.manual_seed(dim)
        x = torch.full((40, dim), 3.0, device=DEV)
        x[1] = -1000.1
        x[2] = 0.0
        x[3:] = 1e4 + torch.randn(37, dim, device=DEV, generator=g)
        y, mean, rstd = forward(L, x, None, None)
        check_forward(x, None, None, y, mean, rstd)
        assert (y[2] == 0).all() and abs(mean[0].item() - 3.0) <= 3.0 * ref.U * 2


def test_nan_and_infinity_stay_in_their_rows():
    L = qb()
    for dim in (100, 1500, 4096, 17000):
        x, gamma, beta, dy = data(6, dim, F32, F32, dim)
        clean, mean, rstd = forward(L, x, gamma, beta)
        bad = x.clone()
        bad[1, dim // 2] = float("nan")
        bad[4, 3] = float("inf")
        y, m, r = forward(L, bad, gamma, beta)
        keep = torch.tensor([0, 2, 3, 5], device=DEV)
        assert torch.equal(y[keep], clean[keep]) and y[1].isnan().all() and y[4].isnan().all()
        dx, dg, db = backward(L, bad, gamma, dy, m, r, F32)
        want = backward(L, x, gamma, dy, mean, rstd, F32)
        assert torch.equal(dx[keep], want[0][keep]) and dx[1].isnan().all()
        assert dg.isnan().all() and torch.equal(db, want[2])


def test_gradient_by_differences():
    """dx, dgamma and dbeta of f = sum(dy * y) against central differences in binary64."""
    L = qb()
    n, dim, step = 5, 70, 1e-6
    x, gamma, beta, dy = data(n, dim, F32, F32, 11)
    _, mean, rstd = forward(L, x, gamma, beta)
    got = [ref.f64(t) for t in backward(L, x, gamma, dy, mean, rstd, F32)]
    args = [ref.f64(x), ref.f64(gamma), ref.f64(beta)]
    d = ref.f64(dy)

    def f(a):
        h, *_ = ref.normalized(a[0], float(np.float32(EPS)), True)
        return (d * (h * a[1] + a[2])).sum()

    for k, g in enumerate(got):
        num = np.zeros_like(args[k])
        for i in np.ndindex(num.shape):
            a = [v.copy() for v in args]
            a[k][i] += step
            up = f(a)
            a[k][i] -= 2 * step
            num[i] = (up - f(a)) / (2 * step)
        # differences: truncation ~ step^2 and cancellation ~ 2^-53 |f| / step; binary32: 1e-5 of the largest
        assert np.abs(num - g).max() <= 1e-5 * np.abs(num).max() + 1e-8
