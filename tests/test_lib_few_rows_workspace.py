"""Workspaces of the gradients of few rows (CPU): not the transposed weights where no kernel writes them, and
never less for more rows, inputs or outputs around the sizes where that changes."""
import random

import pytest

F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def sizes():
    from bit_optimizer_states_amd import binding
    L = binding.lib()
    return {1: L.qb_dequant_linear_backward_workspace_bytes, 2: L.qb_dequant_gated_backward_workspace_bytes}


@pytest.mark.parametrize("count", [1, 2])
@pytest.mark.parametrize("xdt", [F16, BF16])
def test_no_transposed_weights_for_few_rows(sizes, count, xdt):
    """Up to 48 rows dz, the partial sums (16 times dx) and those of the bias's gradient remain; up to 64 rows the
    weights of a layer of 2^24 are the most."""
    for K, N in ((4096, 11008), (4096, 4096), (11008, 4096), (64, 100000)):
        for M in (1, 16, 48, 49, 64):
            rest = M * count * (N + 64) * 2 + 16 * M * K * 4 + (M + 7) // 8 * N * 4 + 3 * 256
            if M > 48:
                rest += min(K * count * (N + 64), (1 << 24) + 64 * K * count) * 2
            assert sizes[count](xdt, M, K, N) <= rest, (M, K, N)


@pytest.mark.parametrize("count", [1, 2])
@pytest.mark.parametrize("xdt", [F32, F16, BF16])
def test_never_less_for_more(sizes, count, xdt):
    f = sizes[count]
    ms = [0, 1, 2, 15, 47, 48, 49, 50, 63, 64, 65, 66]
    ks = [32, 64, 4064, 4096, 4128, 11008, 327680, 327712, 436896, 436928, 445632, (1 << 21) - 32]
    ns = [1, 2, 63, 64, 65, 1000, 2047, 2048, 2049, 4095, 4096, 4097, 11008, 262144, 262145, (1 << 21) - 1]
    for k in ks:
        for n in ns:
            row = [f(xdt, m, k, n) for m in ms]
            assert row == sorted(row), (k, n)
    for m in ms:
        for n in ns:
            row = [f(xdt, m, k, n) for k in ks]
            assert row == sorted(row), (m, n)
        for k in ks:
            row = [f(xdt, m, k, n) for n in ns]
            assert row == sorted(row), (m, k)
    rng = random.Random(7)
    for _ in range(20000):
        m, k = rng.randrange(40, 70), 32 * int(2 ** rng.uniform(0, 12))
        n = max(1, (1 << 24) // (k * count) + rng.randrange(-70, 70))
        assert f(xdt, m, k, n) <= f(xdt, m + rng.randrange(3), k + 32 * rng.randrange(3), n + rng.randrange(80)), (m, k, n)
