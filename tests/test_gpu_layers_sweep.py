"""GPU: the combinations of types and row lengths of the row-wise layers that the
other test files do not reach, so that every compiled instantiation runs; small
token counts, against the same binary64 formulas."""
import pytest
import torch

from gpu_helpers import DEV, qb
from test_gpu_embedding import check_grad, make_ids, normal
from test_gpu_layer_norm import backward as norm_backward
from test_gpu_layer_norm import check_backward as check_norm_backward
from test_gpu_layer_norm import check_forward as check_norm_forward
from test_gpu_layer_norm import data, forward
from test_gpu_stable_embedding import EPS, backward, check_backward, check_forward, weights

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]
# one whole and one ragged length for every way that a row is spread over threads, and a short row
DIMS = [5, 96, 99, 504, 509, 1000, 1003, 1600, 1603, 2048, 2051, 4096, 4099, 8192, 8195, 16384, 16381]


@pytest.mark.parametrize("tdt", TYPES)
@pytest.mark.parametrize("ydt", TYPES)
@pytest.mark.parametrize("own_weights", [False, True])
def test_stable_forward(tdt, ydt, own_weights):
    L = qb()
    wdt = tdt if own_weights else F32
    for dim in DIMS:
        table = normal((6, dim), dim, 0.05, tdt)
        gamma, beta = weights(dim, wdt, dim)
        ids = make_ids(11, 6, dim, torch.int64)
        y = torch.empty(11, dim, dtype=ydt, device=DEV)
        L.qb_stable_embedding(table, ids, gamma, beta, EPS, y, scale=0.9)
        check_forward(table, ids, gamma, beta, 0.9, y)


@pytest.mark.parametrize("gdt", TYPES)
@pytest.mark.parametrize("tdt", TYPES)
@pytest.mark.parametrize("n", [11, 140])
def test_stable_backward(gdt, tdt, n):
    """Few tokens, and enough for the ordering (with long ids among them)."""
    L = qb()
    for dim in DIMS:
        if dim in (96, 99, 1000, 1003):          # the same kernels as 504, 509, 1600, 1603
            continue
        table = normal((6, dim), dim, 0.05, tdt)
        gamma, _ = weights(dim, F32, dim)
        ids = make_ids(n, 6, dim, torch.int32, "zipf")
        dy = normal((n, dim), 3, 0.01, gdt)
        out = backward(L, dy, table, ids, gamma, 1.0, gdt, F32)
        check_backward(dy, table, ids, gamma, 1.0, *out)


@pytest.mark.parametrize("gdt", TYPES)
def test_table_gradient_of_short_rows(gdt):
    L = qb()
    for n, rows, dim in ((300, 40, 5), (300, 3, 1), (7, 40, 7)):
        dy = normal((n, dim), 3, 0.1, gdt)
        ids = make_ids(n, rows, dim, torch.int64, "mixed")
        ws = torch.empty(L.qb_embedding_workspace_bytes(n, rows, dim), dtype=torch.uint8, device=DEV)
        out = torch.empty(rows, dim, dtype=gdt, device=DEV)
        L.qb_embedding_backward(dy, ids, out, ws)
        check_grad(dy, ids, rows, 1.0, gdt, out)


@pytest.mark.parametrize("xdt,wdt", [(F32, F32), (F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)])
def test_layer_norm(xdt, wdt):
    L = qb()
    for dim in DIMS:
        x, gamma, beta, dy = data(5, dim, xdt, wdt, dim)
        y, mean, rstd = forward(L, x, gamma, beta)
        check_norm_forward(x, gamma, beta, y, mean, rstd)
        check_norm_backward(x, gamma, dy, mean, rstd, *norm_backward(L, x, gamma, dy, mean, rstd, wdt))
