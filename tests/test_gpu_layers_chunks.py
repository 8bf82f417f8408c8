"""GPU: the table's gradient on either side of the sizes where its chunks of
ordered tokens go from 16 to 32 (12 waves of 512 columns a CU), with ids of one
token, of about a chunk and of many chunks; whole-numbered dy, so that every sum is
exact, and a workspace of exactly the size asked for."""
import pytest
import torch

from gpu_helpers import DEV, qb
from test_gpu_embedding import BF16, F32, gen

pytestmark = pytest.mark.gpu


def tokens(n, rows, dim, dt, seed):
    g = gen(seed)
    ids = torch.randint(0, rows, (n,), device=DEV, generator=g)
    ids[::11] = rows - 1                                # many chunks
    for k, v in enumerate((14, 15, 16, 17, 18, 31, 32, 33, 34)):
        ids[ids == k] = 20
        ids[torch.randperm(n, device=DEV, generator=g)[:v]] = k
    ids[::13] = -1
    return ids, torch.randint(-2, 3, (n, dim), device=DEV, generator=g).to(dt)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n,dim", [(49152, 40), (49153, 40), (24576, 1001), (24577, 1001), (16384, 1536), (16385, 1536),
                                   (6144, 4096), (6145, 4096), (130000, 24), (20000, 2051)])
def test_table_gradient(n, dim, dt):
    L = qb()
    rows = 700
    ids, dy = tokens(n, rows, dim, dt, n + dim)
    used = ids >= 0
    want = torch.zeros(rows, dim, dtype=torch.float64, device=DEV).index_add_(0, ids[used], dy[used].double())
    size = L.qb_embedding_workspace_bytes(n, rows, dim)
    ws = torch.full((size + 4096,), 0xCD, dtype=torch.uint8, device=DEV)
    out = torch.full((rows, dim), 7.0, device=DEV)
    L.qb_embedding_backward(dy, ids, out, ws[:size])
    torch.cuda.synchronize()
    assert torch.equal(out.double(), want)
    assert (ws[size:] == 0xCD).all()
    # the stable embedding's dbeta is the column sum of the same sums
    size = L.qb_stable_embedding_workspace_bytes(n, rows, dim)
    ws = torch.full((size + 4096,), 0xCD, dtype=torch.uint8, device=DEV)
    table = torch.randn(rows, dim, device=DEV, generator=gen(1))
    dbeta = torch.full((dim,), 7.0, device=DEV)
    L.qb_stable_embedding_backward(dy, table, ids, None, 1e-5, out, None, dbeta, ws[:size])
    torch.cuda.synchronize()
    assert torch.equal(dbeta.double(), want.sum(0))
    assert (ws[size:] == 0xCD).all()
