"""Host: the workspaces of the row-wise layers never shrink when tokens, rows or
elements are added, so that one workspace sized for the largest batch serves every
smaller one (a ragged last batch).  No GPU needed."""
import random

import pytest


@pytest.fixture(scope="module")
def L():
    from bit_optimizer_states_amd import binding
    return binding.lib()


# around every size where a kernel's form changes: the direct gradients (128 tokens), chunks of 16 or 32
# tokens (12 waves a CU), partial rows (256 and 512 workgroups), and powers of two
TOKENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 130, 255, 256, 257, 511, 512, 513, 1535, 1536, 1537, 1552, 1553,
          4095, 6143, 6144, 6145, 8191, 8192, 8193, 12287, 12288, 12289, 16383, 16384, 16385, 24575, 24576, 24577, 30000,
          32767, 32768, 49151, 49152, 49153, 65536, 100000, 1 << 20, (1 << 20) + 1, (1 << 24) - 1, 1 << 24, 1 << 30]
ROWS = [0, 1, 2, 5, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1000, 32000, 128000, 255999, 256000, 256001, 512000,
        512001, (1 << 24) - 1, 1 << 24, 1 << 26]
DIMS = [1, 7, 8, 9, 64, 504, 511, 512, 513, 520, 1024, 1025, 2048, 2049, 4096, 4097, 8192, 8193, 16384]


@pytest.mark.parametrize("name", ["qb_embedding_workspace_bytes", "qb_stable_embedding_workspace_bytes"])
def test_gradient_workspaces_never_shrink(L, name):
    f = getattr(L, name)
    for rows in ROWS:
        for dim in DIMS:
            sizes = [f(n, rows, dim) for n in TOKENS]
            assert sizes[0] > 0 and sizes == sorted(sizes), (rows, dim, sizes)
    for n in TOKENS:
        for dim in DIMS:
            sizes = [f(n, rows, dim) for rows in ROWS]
            assert sizes == sorted(sizes), (n, dim, sizes)
        for rows in ROWS:
            sizes = [f(n, rows, dim) for dim in DIMS]
            assert sizes == sorted(sizes), (n, rows, sizes)


@pytest.mark.parametrize("name", ["qb_embedding_workspace_bytes", "qb_stable_embedding_workspace_bytes"])
def test_gradient_workspaces_never_shrink_in_any_direction(L, name):
    f = getattr(L, name)
    rng = random.Random(5)
    for _ in range(20000):
        small = [int(2 ** rng.uniform(0, b)) for b in (22, 25, 14)]
        large = [min(v + int(2 ** rng.uniform(-2, b - 4)), m) for v, b, m in zip(small, (22, 25, 14), (1 << 30, 1 << 26, 16384))]
        assert 0 < f(*small) <= f(*large), (small, large)


def test_layer_norm_workspace_never_shrinks(L):
    for dim in DIMS + [16385, 40000]:
        sizes = [L.qb_layer_norm_workspace_bytes(n, dim) for n in TOKENS]
        assert sizes[0] > 0 and sizes == sorted(sizes), dim
    for n in TOKENS:
        sizes = [L.qb_layer_norm_workspace_bytes(n, dim) for dim in DIMS + [16385, 40000]]
        assert sizes == sorted(sizes), n
