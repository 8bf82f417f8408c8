"""GPU: the stable embedding (layer norm of an embedding's rows) and its
gradients against the binary64 formulas; the layers' calls in a row, on other
streams and in captured graphs; and one training step of a stable embedding with
the optimizer."""
import numpy as np
import pytest
import torch

import layers_reference as ref
import oracle
from gpu_helpers import DEV, qb
from test_gpu_embedding import lookup, make_ids, normal

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-5


def weights(dim, wdt, seed):
    return (1 + normal((dim,), seed, 0.2)).to(wdt), normal((dim,), seed + 1, 0.2, wdt)


def check_forward(table, ids, gamma, beta, scale, y):
    x = lookup(table, ids, scale, F32)
    want, err, *_ = ref.layer_norm(ref.f64(x), None if gamma is None else ref.f64(gamma),
                                   None if beta is None else ref.f64(beta), float(np.float32(EPS)), table.dtype == F32)
    out = ((ids < 0) | (ids >= table.shape[0])).cpu().numpy()
    want[out], err[out] = 0, 0
    ref.assert_close(y, want, err, f"y {list(y.shape)}")


def check_backward(dy, table, ids, gamma, scale, dtable, dgamma, dbeta, padding_id=-1, old=None):
    rows, dim = table.shape
    s, e_s, k = ref.token_sums(ref.f64(dy), ids.tolist(), rows)
    x = ref.f64(table.float() * torch.tensor(scale, dtype=F32, device=DEV))
    h, _, rstd, e_h, _, e_r = ref.normalized(x, float(np.float32(EPS)), table.dtype == F32)
    g = np.ones(dim) if gamma is None else ref.f64(gamma)
    want, err = ref.norm_grad(s, e_s, h, e_h, rstd, e_r, g)
    sc = abs(float(np.float32(scale)))
    want, err = want * float(np.float32(scale)), err * sc + ref.U * np.abs(want) * sc
    if padding_id >= 0:
        want[padding_id], err[padding_id] = 0, 0
    if old is not None:
        want = want + ref.f64(old[0])
        err = err + ref.U * (np.abs(want) + err)
        still = k == 0
        if padding_id >= 0:
            still[padding_id] = True
        still = torch.from_numpy(still)
        assert torch.equal(dtable[still], old[0][still])
    ref.assert_close(dtable, want, err, f"dtable {list(dtable.shape)}")
    for i, (got, terms, e) in enumerate(((dgamma, s * h, e_s * np.abs(h) + np.abs(s) * e_h), (dbeta, s, e_s))):
        if got is None:
            continue
        want, err = ref.column_sum(terms, e)
        if old is not None:
            want = want + ref.f64(old[1 + i])
            err = err + ref.U * np.abs(want)
        ref.assert_close(got, want, err, ("dgamma", "dbeta")[i])


def backward(L, dy, table, ids, gamma, scale, ddt, wdt, **kw):
    n, (rows, dim) = ids.numel(), table.shape
    ws = torch.full((L.qb_stable_embedding_workspace_bytes(n, rows, dim),), 0xCD, dtype=torch.uint8, device=DEV)
    buf = torch.full((rows + 2, dim), 7.0, dtype=ddt, device=DEV)
    dg, db = (torch.full((dim + 8,), 7.0, dtype=wdt, device=DEV) for _ in range(2))
    L.qb_stable_embedding_backward(dy, table, ids, gamma, EPS, buf[:rows], dg[:dim], db[:dim], ws, scale=scale, **kw)
    torch.cuda.synchronize()
    assert (buf[rows:] == 7.0).all() and (dg[dim:] == 7.0).all() and (db[dim:] == 7.0).all()
    return buf[:rows], dg[:dim], db[:dim]


@pytest.mark.parametrize("tdt,ydt,ddt,wdt", [(F32, F32, F32, F32), (F32, BF16, BF16, F32), (BF16, BF16, BF16, BF16),
                                             (F16, F16, F32, F16), (BF16, F32, F32, F32), (F16, BF16, F16, F32),
                                             (F32, F16, F16, F32), (BF16, F16, BF16, BF16), (F16, F32, F32, F16)])
@pytest.mark.parametrize("n,rows,dim,kind", [(1, 1, 1, "uniform"), (40, 9, 7, "mixed"), (300, 60, 64, "zipf"),
                                             (200, 300, 500, "mixed"), (333, 40, 1001, "zipf"), (200, 20, 2048, "one"),
                                             (64, 11, 4096, "mixed"), (50, 30, 2050, "uniform"), (41, 7, 8192, "mixed"),
                                             (30, 5, 5003, "uniform"), (9, 3, 16384, "mixed"), (70, 4, 9001, "one"),
                                             (128, 40, 264, "zipf"), (129, 40, 264, "zipf"), (200, 5, 8192, "zipf"),
                                             (150, 3, 16384, "zipf"), (140, 9, 5003, "one")])
def test_forward_and_backward(tdt, ydt, ddt, wdt, n, rows, dim, kind):
    L = qb()
    idt = torch.int32 if n % 2 else torch.int64
    table = normal((rows, dim), n + dim, 0.05, tdt)
    gamma, beta = weights(dim, wdt, dim)
    ids = make_ids(n, rows, n, idt, kind)
    y = torch.full((n + 1, dim), 7.0, dtype=ydt, device=DEV)
    L.qb_stable_embedding(table, ids, gamma, beta, EPS, y[:n], scale=1.7)
    torch.cuda.synchronize()
    assert (y[n:] == 7.0).all()
    check_forward(table, ids, gamma, beta, 1.7, y[:n])
    dy = normal((n, dim), 3, 0.01, ydt)
    out = backward(L, dy, table, ids, gamma, 1.7, ddt, wdt)
    check_backward(dy, table, ids, gamma, 1.7, *out)
    again = backward(L, dy, table, ids, gamma, 1.7, ddt, wdt)
    assert all(torch.equal(a, b) for a, b in zip(out, again))


def test_options_of_the_backward_pass():
    """No gamma, a padding id, accumulation, gradients left out."""
    for n in (400, 90):
        options_of_the_backward_pass(qb(), n)


def options_of_the_backward_pass(L, n):
    rows, dim = 70, 333
    table = normal((rows, dim), 1, 0.05, BF16)
    gamma, beta = weights(dim, F32, 2)
    ids = make_ids(n, rows, 4, torch.int64, "zipf")
    pad = int(ids[0])
    dy = normal((n, dim), 5, 0.01, BF16)
    y = torch.empty(n, dim, dtype=BF16, device=DEV)
    for g, b in ((None, None), (gamma, None), (None, beta)):
        L.qb_stable_embedding(table, ids, g, b, EPS, y)
        check_forward(table, ids, g, b, 1.0, y)
    out = backward(L, dy, table, ids, None, 1.0, BF16, F32)
    check_backward(dy, table, ids, None, 1.0, *out)
    out = backward(L, dy, table, ids, gamma, 1.0, F32, F32, padding_id=pad)
    check_backward(dy, table, ids, gamma, 1.0, *out, padding_id=pad)
    assert (out[0][pad] == 0).all()
    ws = torch.empty(L.qb_stable_embedding_workspace_bytes(n, rows, dim), dtype=torch.uint8, device=DEV)
    for p in (-1, pad):
        old = [normal((rows, dim), 6, 1.0, BF16), normal((dim,), 7), normal((dim,), 8)]
        new = [t.clone() for t in old]
        L.qb_stable_embedding_backward(dy, table, ids, gamma, EPS, *new, ws, padding_id=p, accumulate=True)
        check_backward(dy, table, ids, gamma, 1.0, *new, padding_id=p, old=old)
    for keep in ((0, 1), (1, 0), (0, 0)):
        got = [torch.empty_like(t) if k else None for t, k in zip(out[1:], keep)]
        dtable = torch.empty_like(out[0])
        L.qb_stable_embedding_backward(dy, table, ids, gamma, EPS, dtable, *got, ws, padding_id=pad)
        assert torch.equal(dtable, out[0]) and all(g is None or torch.equal(g, t) for g, t in zip(got, out[1:]))


def test_no_tokens_no_rows_and_foreign_ids():
    L = qb()
    rows, dim = 20, 100
    table = normal((rows, dim), 1, 0.05)
    gamma, beta = weights(dim, F32, 2)
    ws = torch.empty(L.qb_stable_embedding_workspace_bytes(50, rows, dim), dtype=torch.uint8, device=DEV)
    none, noid = torch.empty(0, dim, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    out = [torch.full((rows, dim), 7.0, device=DEV), torch.full((dim,), 7.0, device=DEV), torch.full((dim,), 7.0, device=DEV)]
    L.qb_stable_embedding_backward(none, table, noid, gamma, EPS, *out, ws, accumulate=True)
    assert all((t == 7.0).all() for t in out)
    L.qb_stable_embedding_backward(none, table, noid, gamma, EPS, *out, ws)
    assert all((t == 0).all() for t in out)
    ids = torch.full((50,), -1, device=DEV)
    ids[25:] = rows
    dy = torch.full((50, dim), float("nan"), device=DEV)
    out[0].fill_(7.0)
    L.qb_stable_embedding_backward(dy, table, ids, gamma, EPS, *out, ws)
    assert all((t == 0).all() for t in out)
    y = torch.full((50, dim), 7.0, device=DEV)
    L.qb_stable_embedding(table, ids, gamma, beta, EPS, y)
    assert (y == 0).all()
    # an empty table
    empty = torch.empty(0, dim, device=DEV)
    y.fill_(7.0)
    L.qb_stable_embedding(empty, ids, gamma, beta, EPS, y)
    assert (y == 0).all()
    out[1].fill_(7.0)
    L.qb_stable_embedding_backward(dy, empty, ids, gamma, EPS, empty.clone(), out[1], out[2], ws)
    assert (out[1] == 0).all() and (out[2] == 0).all()


def test_equals_lookup_then_layer_norm_in_binary32():
    """The fused call and the two calls in a row, whose lookup is not rounded in binary32: the same bits."""
    L = qb()
    for n, rows, dim in ((50, 30, 100), (33, 9, 1001), (20, 10, 4096)):
        table = normal((rows, dim), 1, 0.05)
        gamma, beta = weights(dim, F32, 2)
        ids = torch.randint(0, rows, (n,), device=DEV)
        x, y, z = (torch.empty(n, dim, device=DEV) for _ in range(3))
        L.qb_embedding(table, ids, x, scale=3.0)
        L.qb_layer_norm(x, gamma, beta, EPS, y)
        L.qb_stable_embedding(table, ids, gamma, beta, EPS, z, scale=3.0)
        assert torch.equal(y, z)


def step_buffers(n, rows, dim, seed):
    table = normal((rows, dim), seed, 0.05)
    gamma, beta = weights(dim, F32, seed + 1)
    ids = make_ids(n, rows, seed, torch.int64, "zipf")
    dy = normal((n, dim), seed + 2, 0.01, BF16)
    L = qb()
    return dict(table=table, gamma=gamma, beta=beta, ids=ids, dy=dy, y=torch.zeros(n, dim, dtype=BF16, device=DEV),
                x=torch.zeros(n, dim, dtype=BF16, device=DEV), z=torch.zeros(n, dim, dtype=BF16, device=DEV),
                mean=torch.zeros(n, device=DEV), rstd=torch.zeros(n, device=DEV),
                dx=torch.zeros(n, dim, dtype=BF16, device=DEV),
                g=[torch.zeros(rows, dim, dtype=BF16, device=DEV), torch.zeros(dim, device=DEV), torch.zeros(dim, device=DEV)],
                h=[torch.zeros(rows, dim, device=DEV), torch.zeros(dim, device=DEV), torch.zeros(dim, device=DEV)],
                ws=[torch.zeros(max(L.qb_stable_embedding_workspace_bytes(n, rows, dim),
                                    L.qb_layer_norm_workspace_bytes(n, dim)), dtype=torch.uint8, device=DEV)
                    for _ in range(3)])


def run_layers(L, b):
    """Both ways through the layers: fused, and lookup + layer norm."""
    L.qb_stable_embedding(b["table"], b["ids"], b["gamma"], b["beta"], EPS, b["y"])
    L.qb_stable_embedding_backward(b["dy"], b["table"], b["ids"], b["gamma"], EPS, *b["g"], b["ws"][0])
    L.qb_embedding(b["table"], b["ids"], b["x"])
    L.qb_layer_norm(b["x"], b["gamma"], b["beta"], EPS, b["z"], mean=b["mean"], rstd=b["rstd"])
    L.qb_layer_norm_backward(b["dy"], b["x"], b["gamma"], b["mean"], b["rstd"], b["dx"], b["h"][1], b["h"][2], b["ws"][1])
    L.qb_embedding_backward(b["dx"], b["ids"], b["h"][0], b["ws"][2])


def outputs(b):
    return [b["y"], b["x"], b["z"], b["mean"], b["rstd"], b["dx"], *b["g"], *b["h"]]


def test_captured_and_replayed():
    """Two graphs with a workspace each: every replay equals the eager result on
    the inputs it finds, with eager calls and new inputs in between."""
    L = qb()
    sets = [step_buffers(700, 150, 520, 1), step_buffers(260, 90, 1001, 50)]
    for b in sets:
        run_layers(L, b)                                # loads every kernel before the capture
    torch.cuda.synchronize()
    graphs = []
    for b in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run_layers(L, b)
        graphs.append(g)
    for turn in range(4):
        for b in sets:
            b["dy"].copy_(normal(b["dy"].shape, 100 + turn, 0.01, BF16))
            b["ids"].copy_(make_ids(b["ids"].numel(), b["table"].shape[0], 200 + turn, torch.int64,
                                    ("one", "mixed", "zipf", "uniform")[turn]))
            for t in outputs(b):
                t.fill_(-3.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for b in sets:
            got = [t.clone() for t in outputs(b)]
            for t in outputs(b):
                t.fill_(5.0)
            run_layers(L, b)
            torch.cuda.synchronize()
            assert all(torch.equal(a, t) for a, t in zip(got, outputs(b))), turn


def test_streams_with_a_workspace_each():
    """Calls that overlap on two streams, each with its own workspace, equal calls in a row."""
    L = qb()
    sets = [step_buffers(900, 300, 768, 1), step_buffers(900, 300, 768, 9)]
    want = []
    for b in sets:
        run_layers(L, b)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outputs(b)])
        for t in outputs(b):
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for b, s in zip(sets, streams):
            with torch.cuda.stream(s):
                run_layers(L, b)
    torch.cuda.synchronize()
    for b, w in zip(sets, want):
        assert all(torch.equal(a, t) for a, t in zip(w, outputs(b)))


def test_training_steps_of_a_stable_embedding_with_the_optimizer():
    """ids -> stable embedding -> a loss -> its gradients -> the multi-tensor AdamW
    step with the policy's states (32 bits for the table, 8 bits for a projection),
    three steps, against the same steps in binary64 on the step's own gradients:
    the table's gradient and parameters stay within binary32 of them."""
    L = qb()
    from bit_optimizer_states_amd import state
    n, rows, dim = 512, 200, 256
    table = normal((rows, dim), 1, 0.05)
    gamma, beta = weights(dim, F32, 2)
    proj = normal((64, dim), 3, 0.05)
    params = [table, gamma, beta, proj]
    states = state.allocate(params, L.QB_ADAMW, blocksize=256, force_32bit=(0,))
    assert states[0][2] is None and states[3][2] is not None          # 32-bit table, 8-bit projection
    grads = [torch.empty_like(p) for p in params]
    tab = L.tensor_table([(p, g, s[0], s[1], s[2], s[3]) for p, g, s in zip(params, grads, states)])
    ws = torch.empty(L.qb_stable_embedding_workspace_bytes(n, rows, dim), dtype=torch.uint8, device=DEV)
    p64 = ref.f64(table).copy()
    m64, v64 = np.zeros_like(p64), np.zeros_like(p64)
    lr, b1, b2, eps, wd = 1e-2, 0.9, 0.999, 1e-8, 0.01
    for step in (1, 2, 3):
        ids = make_ids(n, rows, 10 + step, torch.int64, "zipf")
        y = torch.empty(n, dim, device=DEV)
        L.qb_stable_embedding(table, ids, gamma, beta, EPS, y)
        target = normal((n, 64), 20 + step)
        err = (y @ proj.t() - target) / n                            # loss: half the mean squared error
        grads[3].copy_(err.t() @ y)
        dy = (err @ proj).contiguous()
        L.qb_stable_embedding_backward(dy, table, ids, gamma, EPS, grads[0], grads[1], grads[2], ws)
        check_backward(dy, table, ids, gamma, 1.0, grads[0], grads[1], grads[2])
        hp = L.optim_hparams(L.QB_ADAMW, lr, b1, b2, eps, wd, step=step)
        wsb = torch.empty(L.qb_optimizer_workspace_bytes(hp, tab, 4, 256), dtype=torch.uint8, device=DEV)
        L.qb_multi_tensor_optimizer_step(hp, tab, 4, L.QB_F32, 256, wsb)
        torch.cuda.synchronize()
        g = ref.f64(grads[0])
        m64 = b1 * m64 + (1 - b1) * g
        v64 = b2 * v64 + (1 - b2) * g * g
        p64 = p64 * (1 - lr * wd) - lr / (1 - b1 ** step) * m64 / (np.sqrt(v64) / np.sqrt(1 - b2 ** step) + eps)
        # one step moves a parameter by at most ~lr; binary32 states and update: a few 2^-24 of it and of p
        assert np.abs(ref.f64(table) - p64).max() <= step * (1e-5 * lr + 4 * ref.U * np.abs(p64).max())
        p64 = ref.f64(table).copy()


def test_quantized_table_then_layer_norm():
    """A 4-bit model's embedding: rows decoded by id, then the norm, equals the same on the dequantized table."""
    L = qb()
    rows, dim, n = 64, 512, 100
    w = normal((rows * dim,), 1, 0.02).cpu().numpy()
    codes, absmax = oracle.quantize(w, oracle.NF4, 64)
    cd, am = torch.from_numpy(codes).to(DEV), torch.from_numpy(absmax).to(DEV)
    full = torch.empty(rows, dim, device=DEV)
    L.qb_dequantize(cd, am, None, L.QB_NF4, 64, rows * dim, full)
    gamma, beta = weights(dim, F32, 2)
    ids = make_ids(n, rows, 3, torch.int32, "uniform")
    x, y, z = (torch.empty(n, dim, device=DEV) for _ in range(3))
    L.qb_dequant_embedding(cd, am, None, L.QB_NF4, 64, rows, ids, x, scale=2.0)
    L.qb_layer_norm(x, gamma, beta, EPS, y)
    L.qb_stable_embedding(full, ids, gamma, beta, EPS, z, scale=2.0)
    assert torch.equal(y, z)
