"""GPU: more tokens than one launch of a lookup holds (2^21 workgroups, one token
each for rows of over 1024 elements): the second launch begins where the first ends."""
import pytest
import torch

import oracle
from gpu_helpers import DEV, qb
from test_gpu_embedding import BF16, F32, gen, normal

pytestmark = pytest.mark.gpu

N, ROWS, DIM = (1 << 21) + 5, 100, 1032


def check(y, ids, table):
    for t in range(0, N, 1 << 19):
        i = ids[t:t + (1 << 19)].long()
        want = table[i.clamp(0, ROWS - 1)] * ((i >= 0) & (i < ROWS))[:, None]
        assert torch.equal(y[t:t + (1 << 19)], want), t


def test_lookups():
    L = qb()
    ids = torch.randint(-1, ROWS, (N,), dtype=torch.int32, device=DEV, generator=gen(1))
    y = torch.full((N, DIM), 7.0, dtype=BF16, device=DEV)
    table = normal((ROWS, DIM), 2, 1.0, BF16)
    L.qb_embedding(table, ids, y)
    check(y, ids, table)
    codes, absmax = oracle.quantize(normal((ROWS * DIM,), 3, 0.02).cpu().numpy(), oracle.NF4, 64)
    cd, am = torch.from_numpy(codes).to(DEV), torch.from_numpy(absmax).to(DEV)
    full = torch.empty(ROWS, DIM, device=DEV)
    L.qb_dequantize(cd, am, None, L.QB_NF4, 64, ROWS * DIM, full)
    y.fill_(7.0)
    L.qb_dequant_embedding(cd, am, None, L.QB_NF4, 64, ROWS, ids, y)
    check(y, ids, full.to(BF16))
