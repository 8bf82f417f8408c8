"""GPU: infinite block constants (and values beyond fp16) in the 4-bit layers: an output is the infinity that
the formula gives, also where the inputs are no multiple of a step, and other outputs are as they were."""
import pytest
import torch

import linear_reference as ref
import oracle
import test_gpu_gated as gated
import test_gpu_linear as linear
from gpu_helpers import DEV, qb

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
INF = float("inf")


def positive(shape, seed, xdt):
    return (ref.normal(shape, seed).abs() + 0.25).to(xdt)


def infinite_block(w, block, constant=INF):
    """The block's codes all of 1.0, its constant as given."""
    code = 0xFF if w.code == oracle.NF4 else 0x77
    w.codes[block * w.blocksize // 2:(block + 1) * w.blocksize // 2] = code
    w.absmax[block] = constant


# rows: every number that a workgroup of the rows kernel takes, and the tiled product (1100)
@pytest.mark.parametrize("M", [1, 6, 12, 30, 45, 60, 150, 1100])
@pytest.mark.parametrize("xdt", [BF16, F16, F32])
@pytest.mark.parametrize("K", [160, 224])
def test_one_infinite_block(M, xdt, K):
    """Blocks of 64 that begin at a whole step of a row: the row's last inputs, and the next row's first ones."""
    L = qb()
    N = 21
    w = gated.pair(N, K, oracle.NF4, 64, False, xdt, 1)
    x = positive((M, K), M, xdt)
    clean = [linear.forward(L, x, v) for v in w]
    # row 0: inputs 128 .. 191 of a row of 160 end in row 1; of 224 lie in row 0
    hit = [0, 1] if K == 160 else [0]
    for v in w:
        infinite_block(v, 2, 1e6 if xdt == F16 else INF)
    others = [n for n in range(N) if n not in hit]
    for v, c in zip(w, clean):
        y = linear.forward(L, x, v)
        assert torch.equal(y[:, hit], torch.full_like(y[:, hit], INF)), y[:, hit]
        assert torch.equal(y[:, others], c[:, others])
    y, g, u = gated.forward(L, x, w, "RELU", keep=True)
    for t in (y, g, u):
        assert (t[:, hit] == INF).all() and t[:, others].isfinite().all()


@pytest.mark.parametrize("M", [1, 16, 40, 64, 150, 1100])
@pytest.mark.parametrize("K", [32, 96, 160, 416])
@pytest.mark.parametrize("xdt", [BF16, F32])
def test_every_constant_infinite(M, K, xdt):
    """Nested constants that are all infinite, weights of one sign."""
    L = qb()
    N = 19
    w = gated.pair(N, K, oracle.FP4, 64, True, xdt, 2, 64)
    for v in w:
        v.codes.fill_(0x77)
        v.dq_parts[0].fill_(255)
        v.dq_parts[1].fill_(INF)
    x = positive((M, K), M, xdt)
    assert (linear.forward(L, x, w[0]) == INF).all()
    assert (linear.forward(L, x.neg(), w[0]) == -INF).all()
    assert all((t == INF).all() for t in gated.forward(L, x, w, "SILU", keep=True))


@pytest.mark.parametrize("M", [1, 30, 64, 150])
@pytest.mark.parametrize("xdt", [BF16, F16, F32])
def test_gradients_through_one_infinite_block(M, xdt):
    L = qb()
    N, K = 21, 160
    w = gated.pair(N, K, oracle.NF4, 64, False, xdt, 3)
    dy = positive((M, N), M, xdt)
    clean = linear.backward(L, dy, w[0])[0]
    for v in w:
        infinite_block(v, 2, 1e6 if xdt == F16 else INF)
    hit = torch.zeros(K, dtype=torch.bool, device=DEV)
    hit[128:160] = True                                  # row 0
    hit[:32] = True                                      # row 1
    dx = linear.backward(L, dy, w[0])[0]
    assert (dx[:, hit] == INF).all() and torch.equal(dx[:, ~hit], clean[:, ~hit])
    one = torch.ones_like(dy)
    dx = gated.backward(L, dy, one, one, w, "RELU")[0]
    assert (dx[:, hit] == INF).all() and dx[:, ~hit].isfinite().all()
