"""GPU: gradients of tables of so many rows that the tokens are dealt into ranges
of ids before they are ordered, on either side of the sizes where that begins:
exact sums of whole numbers, the order of every id's tokens, and the stable
embedding's lists of ids."""
import numpy as np
import pytest
import torch

import layers_reference as ref
from gpu_helpers import DEV, qb
from test_gpu_embedding import F32, gen, normal

pytestmark = pytest.mark.gpu

CASES = [(300007, 49151), (300007, 49152), (300007, 70001), (512001, 1023), (512001, 1024), (700000, 20000),
         (1024001, 129), (1100000, 300), (4200000, 3000)]


def make_ids(n, rows, kind, seed):
    g = gen(seed)
    if kind == "one":
        ids = torch.full((n,), rows - 2, device=DEV)
        ids[::7] = torch.randint(0, rows, (len(ids[::7]),), device=DEV, generator=g)
    elif kind == "few":                                 # neighbours: one range of classes, many tokens each
        ids = torch.randint(0, 40, (n,), device=DEV, generator=g) * 3 + rows // 2
    else:
        ids = (3 * (1 + rows / 3) ** torch.rand(n, device=DEV, generator=g, dtype=torch.float64) - 3).long()
        ids = ids.clamp(0, rows - 1)
        ids[::5] = torch.randint(0, rows, (len(ids[::5]),), device=DEV, generator=g)
    ids[3::50] = -1
    ids[5::90] = rows
    ids[7] = rows - 1
    ids[8] = 0
    return ids


def gradient(L, dy, ids, rows, dim):
    n = ids.numel()
    size = L.qb_embedding_workspace_bytes(n, rows, dim)
    ws = torch.full((size + 1024,), 0xCD, dtype=torch.uint8, device=DEV)
    out = torch.full((rows + 1, dim), 7.0, device=DEV)
    L.qb_embedding_backward(dy, ids, out[:rows], ws[:size])
    torch.cuda.synchronize()
    assert (ws[size:] == 0xCD).all() and (out[rows:] == 7.0).all()
    return out[:rows]


@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("kind", ["mixed", "one", "few"])
@pytest.mark.parametrize("rows,n", CASES)
def test_table_gradient(rows, n, kind, idt):
    L = qb()
    dim = 16
    ids = make_ids(n, rows, kind, n).to(idt)
    found = (ids >= 0) & (ids < rows)
    at = ids[found].long()
    whole = torch.randint(-8, 9, (n, dim), device=DEV, generator=gen(n + 1)).float()
    got = gradient(L, whole, ids, rows, dim)
    want = torch.zeros(rows, dim, dtype=torch.float64, device=DEV).index_add_(0, at, whole[found].double())
    assert torch.equal(got.double(), want)

    # ids of up to 16 tokens are summed in the order of the tokens: the same bits as one by one
    dy = normal((n, dim), n + 2)
    got = gradient(L, dy, ids, rows, dim)
    assert torch.equal(got, gradient(L, dy, ids, rows, dim))
    count = torch.bincount(at, minlength=rows)
    some = (count > 0) & (count <= 16)
    used = some.nonzero().flatten().cpu().numpy()
    place = np.full(rows, -1)
    place[used] = np.arange(len(used))
    acc = np.zeros((len(used), dim), np.float32)
    tokens = found.cpu().numpy()
    terms = dy.cpu().numpy()
    for t, v in enumerate(ids.tolist()):
        if tokens[t] and place[v] >= 0:
            acc[place[v]] += terms[t]
    assert np.array_equal(got[some].cpu().numpy(), acc)


@pytest.mark.parametrize("rows,n", CASES)
def test_stable_embedding_gradient(rows, n):
    L = qb()
    dim = 16
    ids = make_ids(n, rows, "mixed", n + 5)
    found = (ids >= 0) & (ids < rows)
    dy = torch.randint(-8, 9, (n, dim), device=DEV, generator=gen(n + 1)).float()
    table = normal((rows, dim), rows, 0.05)
    size = L.qb_stable_embedding_workspace_bytes(n, rows, dim)
    ws = torch.full((size + 1024,), 0xCD, dtype=torch.uint8, device=DEV)
    dtable = torch.full((rows, dim), 7.0, device=DEV)
    dbeta = torch.full((dim,), 7.0, device=DEV)
    L.qb_stable_embedding_backward(dy, table, ids, None, 1e-5, dtable, None, dbeta, ws[:size])
    torch.cuda.synchronize()
    assert (ws[size:] == 0xCD).all()
    s = torch.zeros(rows, dim, dtype=torch.float64, device=DEV).index_add_(0, ids[found], dy[found].double())
    assert torch.equal(dbeta.double(), s.sum(0))
    used = torch.zeros(rows, dtype=torch.bool, device=DEV)
    used[ids[found]] = True
    assert (dtable[~used] == 0).all()
    h, _, rstd, e_h, _, e_r = ref.normalized(ref.f64(table[used]), float(np.float32(1e-5)), True)
    sums = ref.f64(s[used])
    want, err = ref.norm_grad(sums, np.zeros_like(sums), h, e_h, rstd, e_r, np.ones(dim))
    ref.assert_close(dtable[used], want, err, "dtable")
