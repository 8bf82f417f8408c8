"""GPU: embedding lookup (dense and quantized tables) and the gradient of the
table, against plain forms.  Lookups are bit-exact: the products and roundings
are those of IEEE binary32.  Gradients are binary32 sums, compared with binary64
sums within the error of any order of addition."""
import numpy as np
import pytest
import torch

import layers_reference as ref
import oracle
from gpu_helpers import DEV, qb

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(shape, seed, std=1.0, dtype=F32):
    return (torch.empty(shape, device=DEV).normal_(0, std, generator=gen(seed))).to(dtype)


def make_ids(n, rows, seed, idt=torch.int64, kind="mixed"):
    """Ids with repeats; mixed: some outside the table on either side."""
    g = gen(seed)
    ids = torch.randint(0, max(rows, 1), (n,), device=DEV, generator=g)
    if kind == "zipf":
        ids = (3 * (1 + rows / 3) ** torch.rand(n, device=DEV, generator=g, dtype=torch.float64) - 3).long()
        ids = ids.clamp(0, rows - 1)
    if kind == "one":
        ids = torch.full((n,), rows // 2, device=DEV)
    if kind == "mixed" and n > 3:
        ids[torch.randint(0, n, (max(n // 8, 1),), device=DEV, generator=g)] = -1
        ids[n // 2] = rows
        ids[n // 3] = -100
    if idt == torch.int64 and kind == "mixed" and n > 8:
        ids[7] = (1 << 32) + min(3, rows - 1)           # equal to a valid id in its low 32 bits
    return ids.to(idt)


def lookup(table, ids, scale, ydt):
    ids = ids.long()
    rows = table.shape[0]
    found = (ids >= 0) & (ids < rows)
    x = table.float()[ids.clamp(0, rows - 1)] * torch.tensor(scale, dtype=F32, device=DEV)
    return torch.where(found[:, None], x, 0.0).to(ydt)


def same_bits(a, b):
    """Equal bit for bit (0.0 and -0.0 alike: a zero row has positive zeros, a product may have either)."""
    return torch.equal(a, b)


@pytest.mark.parametrize("tdt", [F32, F16, BF16])
@pytest.mark.parametrize("ydt", [F32, F16, BF16])
@pytest.mark.parametrize("n,rows,dim", [(1, 1, 1), (5, 3, 7), (33, 100, 64), (64, 50, 129), (17, 300, 1000), (9, 40, 2049),
                                        (6, 20, 4096), (3, 5, 10007)])
def test_lookup_bit_exact(tdt, ydt, n, rows, dim):
    L = qb()
    for idt, scale in ((torch.int32, 1.0), (torch.int64, 0.7)):
        table = normal((rows, dim), n + dim, 0.05, tdt)
        ids = make_ids(n, rows, dim, idt)
        y = torch.full((n + 1, dim), 7.0, dtype=ydt, device=DEV)
        L.qb_embedding(table, ids, y[:n], scale=scale)
        torch.cuda.synchronize()
        assert same_bits(y[:n], lookup(table, ids, scale, ydt))
        assert (y[n:] == 7.0).all()                      # nothing behind the last row


def test_lookup_special_values_and_empty():
    L = qb()
    table = torch.tensor([[float("nan"), 1.0, float("inf"), -float("inf"), 65504.0, 1e-8, 3e38, -0.0, 2.0]],
                         device=DEV).repeat(3, 1).contiguous()
    table[1] = torch.arange(9.0, device=DEV)
    ids = torch.tensor([1, 0, 5, -1, 1], device=DEV)
    for ydt in (F32, F16, BF16):
        y = torch.empty(5, 9, dtype=ydt, device=DEV)
        L.qb_embedding(table, ids, y, scale=2.0)
        want = lookup(table, ids, 2.0, ydt)
        assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(want)) and torch.equal(y.isnan(), want.isnan())
        assert (y[2:4] == 0).all()                      # outside the table: zeros, although row 0 holds NaN
    # no rows: zeros, the table is not read
    y = torch.full((5, 9), 7.0, device=DEV)
    L.qb_embedding(torch.empty(0, 9, device=DEV), ids, y)
    assert (y == 0).all()
    # no tokens: nothing happens
    L.qb_embedding(table, ids[:0], y[:0])
    # ids and outputs of any leading shape
    y = torch.empty(2, 2, 9, device=DEV)
    L.qb_embedding(table, torch.tensor([[1, 2], [1, 1]], device=DEV), y)
    assert torch.equal(y[0, 0], table[1])


@pytest.mark.parametrize("code", [oracle.DYN8, oracle.NF4, oracle.FP4])
@pytest.mark.parametrize("nested", [False, True])
@pytest.mark.parametrize("rows,dim,B", [(37, 64, 64), (20, 1000, 64), (33, 129, 128), (50, 7, 64), (3, 1, 64), (9, 4096, 4096),
                                        (11, 2056, 256)])
def test_quantized_lookup_bit_exact(code, nested, rows, dim, B):
    """Equal to dequantizing the whole table and looking the rows up."""
    L = qb()
    total = rows * dim
    w = normal((total,), rows + dim, 0.02).cpu().numpy()
    codes, st = oracle.quantize(w, code, B, double_quant=nested)
    cd = torch.from_numpy(codes).to(DEV)
    if nested:
        dq = L.make_dq(torch.from_numpy(st["c2"]).to(DEV), torch.from_numpy(st["absmax2"]).to(DEV),
                       torch.tensor([st["mu"], 0, 0, 0], dtype=F32, device=DEV), 256)
        keep = torch.from_numpy(st["c2"]).to(DEV), torch.from_numpy(st["absmax2"]).to(DEV), \
            torch.tensor([st["mu"], 0, 0, 0], dtype=F32, device=DEV)
        dq = L.make_dq(*keep, 256)
        absmax = None
    else:
        dq, absmax = None, torch.from_numpy(st).to(DEV)
    table = torch.from_numpy(oracle.dequantize(codes, st, code, B, total, oracle.F32)).to(DEV).view(rows, dim)
    for ydt, idt, scale in ((F32, torch.int64, 1.0), (F16, torch.int32, 3.3), (BF16, torch.int64, 1.0)):
        ids = make_ids(29, rows, dim, idt)
        y = torch.full((30, dim), 7.0, dtype=ydt, device=DEV)
        L.qb_dequant_embedding(cd, absmax, dq, code, B, rows, ids, y[:29], scale=scale)
        torch.cuda.synchronize()
        assert same_bits(y[:29], lookup(table, ids, scale, ydt)), (ydt, scale)
        assert (y[29:] == 7.0).all()


def check_grad(dy, ids, rows, scale, ddt, got, padding_id=-1, old=None):
    s, e, k = ref.token_sums(ref.f64(dy), ids.tolist(), rows)
    sc = float(np.float32(scale))
    want, err = s * sc, (e + ref.U * np.abs(s)) * abs(sc)
    if padding_id >= 0:
        want[padding_id] = 0
        err[padding_id] = 0
    if old is not None:
        want = want + ref.f64(old)
        err = err + ref.U * (np.abs(want) + err)
        still = (k == 0)
        if padding_id >= 0:
            still[padding_id] = True
        assert torch.equal(got[torch.from_numpy(still)], old[torch.from_numpy(still)])
    ref.assert_close(got, want, err, f"dtable {list(got.shape)}")


@pytest.mark.parametrize("gdt,ddt", [(F32, F32), (BF16, BF16), (F16, F16), (BF16, F32), (F32, F16)])
@pytest.mark.parametrize("n,rows,dim,kind", [(1, 1, 1, "uniform"), (5, 3, 7, "mixed"), (700, 300, 64, "zipf"),
                                             (300, 40, 1001, "mixed"), (150, 9, 520, "uniform"), (1000, 50, 72, "one"),
                                             (333, 1000, 513, "zipf"), (40, 6, 4096, "mixed"), (6000, 700, 33, "zipf"),
                                             (128, 40, 2600, "zipf"), (129, 40, 520, "zipf"), (128, 5, 64, "one"),
                                             (64, 300, 100, "mixed"), (65, 2, 9, "uniform")])
def test_table_gradient(gdt, ddt, n, rows, dim, kind):
    L = qb()
    for idt in (torch.int32, torch.int64):
        dy = normal((n, dim), n + dim, 0.1, gdt)
        ids = make_ids(n, rows, n, idt, kind)
        ws = torch.full((L.qb_embedding_workspace_bytes(n, rows, dim),), 0xCD, dtype=torch.uint8, device=DEV)
        buf = torch.full((rows + 2, dim), 7.0, dtype=ddt, device=DEV)
        out = buf[:rows]
        L.qb_embedding_backward(dy, ids, out, ws, scale=0.7)
        torch.cuda.synchronize()
        check_grad(dy, ids, rows, 0.7, ddt, out)
        assert (buf[rows:] == 7.0).all()                 # nothing behind the last row
        # the same bits again, from another state of the workspace
        ws.fill_(0x3C)
        again = torch.empty_like(out)
        L.qb_embedding_backward(dy, ids, again, ws, scale=0.7)
        assert torch.equal(out, again)


@pytest.mark.parametrize("ddt", [F32, F16, BF16])
def test_table_gradient_accumulates_and_skips_padding(ddt):
    for n in (500, 100):
        accumulates_and_skips_padding(qb(), n, ddt)


def accumulates_and_skips_padding(L, n, ddt):
    rows, dim = 90, 201
    dy = normal((n, dim), 1, 0.1, BF16)
    ids = make_ids(n, rows, 2, torch.int64, "zipf")
    pad = int(ids[0])
    ws = torch.empty(L.qb_embedding_workspace_bytes(n, rows, dim), dtype=torch.uint8, device=DEV)
    out = torch.full((rows, dim), 7.0, dtype=ddt, device=DEV)
    L.qb_embedding_backward(dy, ids, out, ws, padding_id=pad)
    check_grad(dy, ids, rows, 1.0, ddt, out, padding_id=pad)
    assert (out[pad] == 0).all()
    old = normal((rows, dim), 3, 1.0, ddt)
    for p in (-1, pad):
        out = old.clone()
        L.qb_embedding_backward(dy, ids, out, ws, padding_id=p, accumulate=True)
        check_grad(dy, ids, rows, 1.0, ddt, out, padding_id=p, old=old)
    # a padding id outside the table skips nothing
    out.zero_()
    L.qb_embedding_backward(dy, ids, out, ws, padding_id=rows + 5)
    check_grad(dy, ids, rows, 1.0, ddt, out)


def test_table_gradient_of_no_tokens_and_of_foreign_ids():
    L = qb()
    rows, dim = 30, 65
    ws = torch.empty(L.qb_embedding_workspace_bytes(100, rows, dim), dtype=torch.uint8, device=DEV)
    out = torch.full((rows, dim), 7.0, device=DEV)
    L.qb_embedding_backward(torch.empty(0, dim, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV), out, ws,
                            accumulate=True)
    assert (out == 7.0).all()
    L.qb_embedding_backward(torch.empty(0, dim, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV), out, ws)
    assert (out == 0).all()
    # every id outside the table; their dy may hold anything
    dy = torch.full((100, dim), float("nan"), device=DEV)
    ids = torch.full((100,), -1, device=DEV)
    ids[50:] = rows
    out.fill_(7.0)
    L.qb_embedding_backward(dy, ids, out, ws)
    assert (out == 0).all()
    # NaN enters the rows whose tokens hold it, and no others
    dy = torch.ones(100, dim, device=DEV)
    dy[3, 5] = float("nan")
    dy[4] = float("inf")
    ids = torch.arange(100, device=DEV) % 10
    L.qb_embedding_backward(dy, ids, out, ws)
    want = torch.zeros(rows, dim, device=DEV)
    want[:10] = 10.0
    want[4] = float("inf")
    want[3, 5] = float("nan")
    assert torch.equal(torch.nan_to_num(out, nan=-5.0), torch.nan_to_num(want, nan=-5.0))


def test_table_gradient_of_large_vocabulary_and_many_tokens():
    """More entries than one class of ids holds, ids of every class, and an id
    with more tokens than a chunk next to ids with few."""
    L = qb()
    n, rows, dim = 30000, 300007, 16
    g = gen(5)
    ids = torch.randint(0, rows, (n,), device=DEV, generator=g)
    ids[::3] = 299999
    ids[1::7] = 0
    dy = torch.randint(-8, 9, (n, dim), device=DEV, generator=g).float()       # sums exact in binary32
    ws = torch.empty(L.qb_embedding_workspace_bytes(n, rows, dim), dtype=torch.uint8, device=DEV)
    out = torch.empty(rows, dim, device=DEV)
    L.qb_embedding_backward(dy, ids, out, ws)
    want = torch.zeros(rows, dim, dtype=torch.float64, device=DEV).index_add_(0, ids, dy.double())
    assert torch.equal(out.double(), want)


def test_offsets_beyond_32_bits():
    """A table and an output of more than 2^32 bytes: the last rows are read and written where they are."""
    L = qb()
    rows, dim = 300000, 8192                      # 4.9 GB
    table = torch.zeros(rows, dim, dtype=BF16, device=DEV)
    table[rows - 3:] = normal((3, dim), 9, 1.0, BF16)
    ids = torch.full((rows,), 5, dtype=torch.int32, device=DEV)
    ids[-2:] = rows - 1
    ids[17] = rows - 3
    y = torch.empty(rows, dim, dtype=BF16, device=DEV)
    L.qb_embedding(table, ids, y)
    assert torch.equal(y[-2:], table[rows - 1:].expand(2, dim)) and torch.equal(y[17], table[rows - 3])
    assert (y[:17] == 0).all() and (y[18:1000] == 0).all() and (y[-1000:-2] == 0).all()
    del y
    dy = torch.zeros(rows, dim, dtype=BF16, device=DEV)
    dy[-2:] = 1.5
    dy[17] = -2.0
    ws = torch.empty(L.qb_embedding_workspace_bytes(rows, rows, dim), dtype=torch.uint8, device=DEV)
    table.fill_(3.0)
    L.qb_embedding_backward(dy, ids, table, ws)
    assert (table[rows - 1] == 3.0).all() and (table[rows - 3] == -2.0).all() and (table[5] == 0).all()
    assert (table[6:2000] == 0).all() and (table[rows - 2] == 0).all()
