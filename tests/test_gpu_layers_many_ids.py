"""GPU: gradients in which a workgroup takes many ids or rows in turn: the
stable embedding's over far more used ids than it has workgroups (512), and over
more than 64 ids a workgroup; layer norm's over more rows of over 16384 elements
than it has partial rows (64)."""
import numpy as np
import pytest
import torch

import layers_reference as ref
from gpu_helpers import DEV, qb
from test_gpu_embedding import BF16, F16, F32, gen, normal
from test_gpu_layer_norm import backward as norm_backward
from test_gpu_layer_norm import data
from test_gpu_stable_embedding import EPS, backward, weights

pytestmark = pytest.mark.gpu


def sums_by_id(dy, ids, rows):
    """S[v], its error (k terms: k u sum |dy|) and the number k of tokens."""
    t, at = torch.from_numpy(dy), torch.from_numpy(ids)
    s = torch.zeros(rows, dy.shape[1], dtype=torch.float64).index_add_(0, at, t).numpy()
    a = torch.zeros(rows, dy.shape[1], dtype=torch.float64).index_add_(0, at, t.abs()).numpy()
    k = np.bincount(ids, minlength=rows).astype(float)
    return s, a * k[:, None] * ref.U, k


def check_columns(got, terms, e_terms, path, what):
    """A sum over the rows of `terms`, at most `path` additions deep."""
    want = terms.sum(0)
    ref.assert_close(got, want, e_terms.sum(0) + path * ref.U * (np.abs(terms) + e_terms).sum(0), what)


@pytest.mark.parametrize("tdt,gdt,ddt,wdt", [(F32, F32, F32, F32), (BF16, BF16, BF16, BF16), (F16, F32, BF16, F32)])
@pytest.mark.parametrize("n,rows,dim", [(6000, 3000, 7), (6000, 3000, 200), (6000, 2500, 1001), (4000, 1800, 4099),
                                        (3000, 1500, 8192), (2500, 1300, 9001), (120000, 40000, 16)])
def test_stable_embedding_gradient(n, rows, dim, tdt, gdt, ddt, wdt):
    L = qb()
    ids = torch.randint(0, rows, (n,), device=DEV, generator=gen(n + dim))
    ids[5::20] = 17                                     # a long id, and tokens of no id
    ids[7::50] = -1
    pad = int(ids[0])
    table = normal((rows, dim), dim, 0.05, tdt)
    gamma, _ = weights(dim, wdt, dim)
    dy = normal((n, dim), 3, 0.01, gdt)
    dtable, dgamma, dbeta = backward(L, dy, table, ids, gamma, 1.7, ddt, wdt, padding_id=pad)
    again = backward(L, dy, table, ids, gamma, 1.7, ddt, wdt, padding_id=pad)
    assert all(torch.equal(a, b) for a, b in zip((dtable, dgamma, dbeta), again))

    keep = ids.cpu().numpy()
    s, e_s, k = sums_by_id(ref.f64(dy)[keep >= 0], keep[keep >= 0], rows)
    used = int((k > 0).sum())
    assert used > 2 * 512 and (n < 100000 or used > 64 * 512)
    x = ref.f64(table.float() * torch.tensor(1.7, dtype=F32, device=DEV))
    h, _, rstd, e_h, _, e_r = ref.normalized(x, float(np.float32(EPS)), True)
    sc = float(np.float32(1.7))
    want, err = ref.norm_grad(s, e_s, h, e_h, rstd, e_r, ref.f64(gamma))
    want, err = want * sc, err * sc + ref.U * np.abs(want) * sc
    want[pad], err[pad] = 0, 0
    ref.assert_close(dtable, want, err, "dtable")
    # a workgroup adds its ids in turn, then 512 / 32 partial rows and 32 sums of these are added
    path = used // 512 + 1 + 16 + 32
    check_columns(dgamma, s * h, e_s * np.abs(h) + np.abs(s) * e_h, path, "dgamma")
    check_columns(dbeta, s, e_s, path, "dbeta")


@pytest.mark.parametrize("n", [65, 150, 400])
@pytest.mark.parametrize("xdt,wdt", [(F32, F32), (BF16, BF16), (F16, F32)])
def test_layer_norm_gradient_of_many_long_rows(n, xdt, wdt):
    L = qb()
    dim = 16387
    x, gamma, _, dy = data(n, dim, xdt, wdt, n)
    xd, d = ref.f64(x), ref.f64(dy)
    m, _, r = ref.statistics(xd, EPS)
    mean, rstd = (torch.from_numpy(v).float().to(DEV) for v in (m, r))
    m, r = ref.f64(mean), ref.f64(rstd)
    dx, dgamma, dbeta = norm_backward(L, x, gamma, dy, mean, rstd, wdt)
    h = (xd - m[:, None]) * r[:, None]
    e_h = 2 * ref.U * np.abs(h)
    want, err = ref.norm_grad(d, np.zeros_like(d), h, e_h, r, np.zeros_like(r), ref.f64(gamma))
    ref.assert_close(dx, want, err, "dx")
    path = -(-n // 64) + 2 + 32                         # rows of a partial row, then 64 / 32 of these and 32 sums
    check_columns(dgamma, d * h, np.abs(d) * e_h, path, "dgamma")
    check_columns(dbeta, d, np.zeros_like(d), path, "dbeta")
