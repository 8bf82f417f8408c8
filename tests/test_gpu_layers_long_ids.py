"""GPU: gradients of tables where a few ids hold most of the tokens (padding, a
batch of one token): their sums are taken by many waves and joined, by one wave
for up to 64 chunks of tokens (a chunk: 16 tokens, 32 from 16384 tokens on), by a
whole workgroup beyond."""
import pytest
import torch

from gpu_helpers import DEV, qb
from test_gpu_embedding import BF16, F32, check_grad, gen, normal
from test_gpu_stable_embedding import backward, check_backward, weights

pytestmark = pytest.mark.gpu

# tokens, table rows, and the tokens of single ids (the others even over the table, a few outside it)
CASES = [(6000, 40, {3: 1500, 0: 1100, 39: 2000}),          # two and more beyond 64 chunks of 16
         (3000, 700, {5: 1024, 6: 1025, 7: 300}),           # about 64 chunks
         (1200, 9, {8: 1200}),                              # all of one id
         (17000, 33, {2: 8000, 32: 2049, 1: 2048, 9: 33})]  # chunks of 32


def ids_of(n, rows, counts, seed):
    g = gen(seed)
    ids = torch.randint(-2, rows + 1, (n,), device=DEV, generator=g)
    at = 0
    for v, k in counts.items():
        ids[ids == v] = -1                                  # exactly k tokens of v
        ids[at:at + k] = v
        at += k
    return ids[torch.randperm(n, device=DEV, generator=g)].contiguous()


@pytest.mark.parametrize("gdt,ddt", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("dim", [7, 200, 1001])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_table_gradient(case, dim, gdt, ddt):
    L = qb()
    n, rows, counts = CASES[case]
    ids = ids_of(n, rows, counts, dim)
    dy = normal((n, dim), dim, 0.1, gdt)
    ws = torch.full((L.qb_embedding_workspace_bytes(n, rows, dim),), 0xCD, dtype=torch.uint8, device=DEV)
    buf = torch.full((rows + 2, dim), 7.0, dtype=ddt, device=DEV)
    L.qb_embedding_backward(dy, ids, buf[:rows], ws, scale=0.7)
    torch.cuda.synchronize()
    check_grad(dy, ids, rows, 0.7, ddt, buf[:rows])
    assert (buf[rows:] == 7.0).all()
    again = torch.empty_like(buf[:rows])
    L.qb_embedding_backward(dy, ids, again, ws, scale=0.7)
    assert torch.equal(buf[:rows], again)
    # a frequent id is padding; added to what is there
    pad = next(iter(counts))
    old = normal((rows, dim), 5, 1.0, ddt)
    out = old.clone()
    L.qb_embedding_backward(dy, ids, out, ws, scale=0.7, padding_id=pad, accumulate=True)
    torch.cuda.synchronize()
    check_grad(dy, ids, rows, 0.7, ddt, out.cpu(), padding_id=pad, old=old.cpu())


@pytest.mark.parametrize("tdt,gdt,ddt,wdt", [(F32, F32, F32, F32), (BF16, BF16, F32, BF16)])
@pytest.mark.parametrize("dim", [7, 200, 1001])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_stable_embedding_gradient(case, dim, tdt, gdt, ddt, wdt):
    L = qb()
    n, rows, counts = CASES[case]
    ids = ids_of(n, rows, counts, dim + 1)
    table = normal((rows, dim), dim, 0.05, tdt)
    gamma, _ = weights(dim, wdt, dim)
    dy = normal((n, dim), 3, 0.01, gdt)
    out = backward(L, dy, table, ids, gamma, 1.7, ddt, wdt)
    check_backward(dy, table, ids, gamma, 1.7, *out)
    again = backward(L, dy, table, ids, gamma, 1.7, ddt, wdt)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
