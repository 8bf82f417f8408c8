"""GPU: the 4-bit linear layer with bias, activation and residual, and its gradients,
against the binary64 formulas within the rounding error of their evaluation
(linear_reference.py)."""
import numpy as np
import pytest
import torch

import linear_reference as ref
import oracle
from gpu_helpers import DEV, qb

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NF4, FP4 = oracle.NF4, oracle.FP4
ACTS = ["NONE", "RELU", "GELU", "GELU_TANH", "SILU"]


def kind_of(L, name):
    return getattr(L, "QB_ACT_" + name)


def workspace(size, extra=256):
    """A workspace of exactly `size` bytes, with a guard behind it."""
    ws = torch.full((size + extra,), 0x5A, dtype=torch.uint8, device=DEV)
    return ws[:size], ws[size:]


def forward(L, x, w, bias=None, act="NONE", residual=None, keep=False, in_place=False):
    m, n = x.shape[0], w.n
    ws, guard = workspace(L.qb_dequant_linear_workspace_bytes(L._DTYPE[x.dtype], m, w.k, n))
    y = torch.full((m + 1, n), 7.0, dtype=x.dtype, device=DEV)
    z = torch.full((m + 1, n), 7.0, dtype=x.dtype, device=DEV) if keep else None
    if in_place:
        y[:m] = residual
        residual = y[:m]
    L.qb_dequant_linear(x, w.codes, w.absmax, w.code, w.blocksize, n, y[:m], ws, bias=bias, act=kind_of(L, act),
                        residual=residual, z=z[:m] if keep else None, dq=w.dq(L))
    torch.cuda.synchronize()
    assert (guard == 0x5A).all() and (y[m:] == 7.0).all() and (z is None or (z[m:] == 7.0).all())
    return (y[:m], z[:m]) if keep else y[:m]


def backward(L, dy, w, z=None, act="NONE", dx=True, dz=False, bias_dt=None, old=None):
    m, n = dy.shape
    ws, guard = workspace(L.qb_dequant_linear_backward_workspace_bytes(L._DTYPE[dy.dtype], m, w.k, n))
    gx = torch.full((m + 1, w.k), 7.0, dtype=dy.dtype, device=DEV)
    gz = torch.full((m + 1, n), 7.0, dtype=dy.dtype, device=DEV)
    gb = None if bias_dt is None else torch.full((n,), 7.0, dtype=bias_dt, device=DEV) if old is None else old.clone()
    L.qb_dequant_linear_backward(dy, w.codes, w.absmax, w.code, w.blocksize, w.k, gx[:m] if dx else None, ws,
                                 act=kind_of(L, act), z=z, dz=gz[:m] if dz else None, dbias=gb,
                                 accumulate=old is not None, dq=w.dq(L))
    torch.cuda.synchronize()
    assert (guard == 0x5A).all() and (gx[m if dx else 0:] == 7.0).all() and (gz[m if dz else 0:] == 7.0).all()
    return gx[:m] if dx else None, gz[:m] if dz else None, gb


def check_forward(L, x, w, bias, act, residual, y, z=None):
    f = ref.f64
    want_z, e_z, want, e = ref.linear(L, f(x), w.w, None if bias is None else f(bias), kind_of(L, act),
                                      None if residual is None else f(residual))
    if z is not None:
        ref.assert_close(z, want_z, e_z, "z")
    ref.assert_close(y, want, e, "y")


def check_backward(L, dy, w, z, act, dx, dz, dbias, old=None):
    d = ref.f64(dy)
    e = np.zeros_like(d)
    if act != "NONE":
        _, slope, _, e_slope = ref.act(L, kind_of(L, act), ref.f64(z))
        e = np.abs(d) * e_slope + ref.U * np.abs(d * slope)
        d = d * slope
    if dz is not None:
        ref.assert_close(dz, d, e, "dz")
    if dx is not None:
        ref.assert_close(dx, *ref.rounded_product(d, e, w.w, dy.dtype), "dx")
    if dbias is not None:
        err = e.sum(0) + (d.shape[0] + 2) * ref.U * (np.abs(d) + e).sum(0)
        want = d.sum(0)
        if old is not None:
            want = want + ref.f64(old)
            err = err + ref.U * (np.abs(want) + err)
        ref.assert_close(dbias, want, err, "dbias")


# rows: the staged ones, each tile count of the small kernel, both sides of 64, tiles of the
# product whole and ragged; inputs: whole and half steps; outputs: odd ones, fewer than a unit
SHAPES = [(1, 4096, 300), (8, 512, 64), (9, 160, 40), (16, 32, 3), (17, 1024, 40), (33, 96, 17), (64, 256, 48),
          (65, 256, 48), (65, 32, 1), (100, 96, 131), (128, 64, 128), (129, 1056, 129), (200, 992, 1001),
          (300, 128, 4), (257, 2048, 520)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("xdt", [BF16, F16, F32])
def test_shapes_and_types(M, K, N, xdt):
    """Everything in the epilogue, the pre-activation kept; then its gradients."""
    L = qb()
    print(f"[linear] {M} {K} {N} {xdt}", flush=True)
    w = ref.Weight(N, K, NF4, 64, False, xdt, seed=M + K + N)
    x, bias, residual = (ref.normal(s, M + i, dtype=xdt) for i, s in enumerate([(M, K), (N,), (M, N)]))
    y, z = forward(L, x, w, bias, "SILU", residual, keep=True)
    check_forward(L, x, w, bias, "SILU", residual, y, z)
    dy = ref.normal((M, N), 5, 0.1, xdt)
    dx, dz, db = backward(L, dy, w, z, "SILU", dz=True, bias_dt=xdt)
    check_backward(L, dy, w, z, "SILU", dx, dz, db)


@pytest.mark.parametrize("M", [7, 40, 150])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("xdt", [BF16, F32])
def test_activations(M, act, xdt):
    L = qb()
    w = ref.Weight(73, 128, FP4, 128, False, xdt, seed=3)
    x = ref.normal((M, 128), 1, 2.0, xdt)
    bias = ref.normal((73,), 2, 3.0)
    y, z = forward(L, x, w, bias, act, keep=True)
    check_forward(L, x, w, bias, act, None, y, z)
    dy = ref.normal((M, 73), 4, 1.0, xdt)
    dx, dz, db = backward(L, dy, w, z if act != "NONE" else None, act, dz=True, bias_dt=F32)
    check_backward(L, dy, w, z, act, dx, dz, db)


@pytest.mark.parametrize("code", [NF4, FP4])
@pytest.mark.parametrize("blocksize", [64, 128, 512, 4096])
@pytest.mark.parametrize("nested", [False, True])
@pytest.mark.parametrize("M", [5, 40, 90])
def test_codes_blocks_and_nesting(code, blocksize, nested, M):
    L = qb()
    w = ref.Weight(200, 1120, code, blocksize, nested, BF16, seed=blocksize + code, blocksize2=64 if M == 5 else 256)
    x = ref.normal((M, 1120), 1, dtype=BF16)
    check_forward(L, x, w, None, "NONE", None, forward(L, x, w))
    dy = ref.normal((M, 200), 2, dtype=BF16)
    check_backward(L, dy, w, None, "NONE", backward(L, dy, w)[0], None, None)


@pytest.mark.parametrize("M", [3, 30, 64, 70, 300])
@pytest.mark.parametrize("xdt", [BF16, F16, F32])
def test_every_weight_in_its_place(M, xdt):
    """Rows of the identity give back the weights themselves, bit for bit, in both directions."""
    L = qb()
    for n, k in ((137, 160), (320, 96), (64, 1024)):
        w = ref.Weight(n, k, NF4, 64, True, xdt, seed=n)
        values = w.values.to(DEV)
        for at in range(0, max(n, k), M):
            rows = torch.arange(at, at + M, device=DEV)
            x = torch.zeros(M, k, dtype=xdt, device=DEV)
            live = rows < k
            x[live, rows[live]] = 1.0
            want = torch.zeros(M, n, dtype=xdt, device=DEV)
            want[live] = values[:, rows[live]].T
            assert torch.equal(forward(L, x, w), want)
            dy = torch.zeros(M, n, dtype=xdt, device=DEV)
            live = rows < n
            dy[live, rows[live]] = 1.0
            want = torch.zeros(M, k, dtype=xdt, device=DEV)
            want[live] = values[rows[live]]
            assert torch.equal(backward(L, dy, w)[0], want)


@pytest.mark.parametrize("M", [12, 130])
@pytest.mark.parametrize("N", [64, 129])
def test_parts_of_the_epilogue(M, N):
    """Each optional input and output with and without the others; the residual in place."""
    L = qb()
    w = ref.Weight(N, 256, NF4, 64, True, BF16, seed=1)
    x, residual, dy = (ref.normal(s, i, dtype=BF16) for i, s in enumerate([(M, 256), (M, N), (M, N)]))
    for bias in (None, ref.normal((N,), 7), ref.normal((N,), 8, dtype=BF16)):
        for res in (None, residual):
            for act in ("NONE", "GELU_TANH"):
                y, z = forward(L, x, w, bias, act, res, keep=True)
                check_forward(L, x, w, bias, act, res, y, z)
                assert torch.equal(forward(L, x, w, bias, act, res), y)
                if res is not None:
                    assert torch.equal(forward(L, x, w, bias, act, res, in_place=True), y)
    for act in ("NONE", "GELU_TANH"):
        dx, dz, db = backward(L, dy, w, z, act, dz=True, bias_dt=F32)
        check_backward(L, dy, w, z, act, dx, dz, db)
        for use_x in (False, True):
            for use_z in (False, True):
                for bias_dt in (None, F32):
                    gx, gz, gb = backward(L, dy, w, z, act, dx=use_x, dz=use_z, bias_dt=bias_dt)
                    assert gx is None or torch.equal(gx, dx)
                    assert gz is None or torch.equal(gz, dz)
                    assert gb is None or torch.equal(gb, db)


@pytest.mark.parametrize("bias_dt", [F32, BF16])
def test_bias_gradient_accumulates(bias_dt):
    L = qb()
    for M, N in ((1, 7), (40, 65), (1000, 33), (70, 1500)):
        w = ref.Weight(N, 32, NF4, 64, False, BF16, seed=1)
        dy, z = ref.normal((M, N), 1, dtype=BF16), ref.normal((M, N), 2, dtype=BF16)
        old = ref.normal((N,), 3, 5.0, bias_dt)
        for act in ("NONE", "SILU"):
            _, _, db = backward(L, dy, w, z, act, dx=False, bias_dt=bias_dt, old=old)
            check_backward(L, dy, w, z, act, None, None, db, old)


def test_no_rows():
    L = qb()
    w = ref.Weight(48, 64, NF4, 64, False, BF16, seed=1)
    x, dy = torch.empty(0, 64, dtype=BF16, device=DEV), torch.empty(0, 48, dtype=BF16, device=DEV)
    forward(L, x, w, keep=True)
    old = ref.normal((48,), 1)
    assert torch.equal(backward(L, dy, w, bias_dt=F32, old=old)[2], old)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    db = torch.full((48,), 7.0, device=DEV)
    L.qb_dequant_linear_backward(dy, w.codes, w.absmax, NF4, 64, 64, None, ws, dbias=db)
    assert (db == 0.0).all()


@pytest.mark.parametrize("M", [20, 100])
def test_infinities_and_nan_stay_in_their_rows(M):
    L = qb()
    w = ref.Weight(80, 96, NF4, 64, False, BF16, seed=1)
    x = ref.normal((M, 96), 1, dtype=BF16)
    clean = forward(L, x, w)
    x[3, 95], x[M - 1, 5] = float("nan"), float("inf")
    y = forward(L, x, w)
    rows = torch.ones(M, dtype=torch.bool)
    rows[[3, M - 1]] = False
    assert torch.equal(y[rows], clean[rows]) and y[3].isnan().all()
    live = (w.values[:, 5] != 0).to(DEV)
    assert y[M - 1][live].isinf().all()
    dy = ref.normal((M, 80), 2, dtype=BF16)
    clean = backward(L, dy, w)[0]
    dy[3, 79], dy[M - 1, 5] = float("nan"), float("inf")
    dx = backward(L, dy, w)[0]
    assert torch.equal(dx[rows], clean[rows]) and dx[3].isnan().all()
    assert dx[M - 1][(w.values[5] != 0).to(DEV)].isinf().all()


def test_large_pre_activations():
    """act and act' where exponentials leave binary32's range: the limits, no NaN."""
    L = qb()
    w = ref.Weight(64, 32, NF4, 64, False, F32, seed=1)
    z = torch.tensor([0.0, 1e-30, -1e-30, 30.0, -30.0, 88.0, -88.0, 104.0, -104.0, 1e4, -1e4, 1e15, -1e15, 1e30, -1e30,
                      3e38, -3e38, 6.0, -6.0, 0.5], device=DEV).repeat(7, 16)[:, :320].contiguous()
    for act in ACTS[1:]:
        bias_w = ref.Weight(320, 32, NF4, 64, False, F32, seed=1)
        x = torch.zeros(7, 32, device=DEV)
        y, kept = forward(L, x, bias_w, z[0].contiguous(), act, keep=True)
        assert torch.equal(kept, z)
        dz = backward(L, torch.ones_like(z), bias_w, z, act, dx=False, dz=True)[1]
        assert y.isfinite().all() and dz.isfinite().all(), act
        small = z.abs().cpu().numpy() < 200
        a, slope, ea, es = ref.act(L, kind_of(L, act), np.where(small, ref.f64(z), 0.0))
        for got, want, err in ((y, a, ea), (dz, slope, es)):
            bad = small & ~(np.abs(ref.f64(got) - want) <= 1.001 * (err + ref.half_step(F32, want)))
            assert not bad.any(), (act, ref.f64(z)[bad][0], ref.f64(got)[bad][0], want[bad][0])
        big = z.abs() > 200
        assert torch.equal(y[big], z[big].clamp_min(0.0)) and torch.equal(dz[big], (z[big] > 0).float()), act
    del w


def test_gradient_against_differences():
    """The binary32 gradient of sum(c * y) against central differences of the forward call."""
    L = qb()
    M, K, N, h = 4, 64, 37, 2.0 ** -7
    w = ref.Weight(N, K, NF4, 64, False, F32, seed=2)
    x, bias, c = ref.normal((M, K), 1), ref.normal((N,), 2), ref.normal((M, N), 3)
    for act in ACTS:
        if act == "RELU":
            continue                                   # (not differentiable where z = 0)
        _, z = forward(L, x, w, bias, act, keep=True)
        dx, _, db = backward(L, c, w, z, act, bias_dt=F32)
        value = lambda x, b: ref.f64(forward(L, x.contiguous(), w, b, act)) @ ref.f64(c).T  # noqa: E731
        for k in (0, 17, 63):
            step = torch.zeros_like(x)
            step[:, k] = h
            d = np.diag(value(x + step, bias) - value(x - step, bias)) / (2 * h)
            # third derivatives of every act stay below 3: h^2 / 6 * 3 sum |c w^3|; the values are off by
            # (K + 40) 2u (|z| + 1) |c| per output
            wk = np.abs(w.w[:, k])
            err = h * h / 2 * (np.abs(ref.f64(c)) @ wk ** 3) + (K + 40) * 2 * ref.U / h * (
                (np.abs(ref.f64(z)) + 8) * np.abs(ref.f64(c))).sum(1)
            assert (np.abs(d - ref.f64(dx)[:, k]) <= err).all(), act
        n = 11
        step = torch.zeros_like(bias)
        step[n] = h
        d = np.trace(value(x, bias + step) - value(x, bias - step)) / (2 * h)
        err = h * h / 2 * np.abs(ref.f64(c)[:, n]).sum() + (K + 40) * 2 * ref.U / h * (
            (np.abs(ref.f64(z)) + 8) * np.abs(ref.f64(c))).sum()
        assert abs(d - float(db[n])) <= err, act


@pytest.mark.parametrize("M", [6, 130])
def test_captured_calls_replay(M):
    """Forward and backward captured into one graph, replayed on new inputs with eager work in between."""
    L = qb()
    K, N = 256, 200
    w = ref.Weight(N, K, NF4, 64, True, BF16, seed=4)
    x, dy, bias = ref.normal((M, K), 1, dtype=BF16), ref.normal((M, N), 2, dtype=BF16), ref.normal((N,), 3)
    y, z, dx = (torch.empty(M, n, dtype=BF16, device=DEV) for n in (N, N, K))
    db = torch.empty(N, device=DEV)
    ws = torch.empty(L.qb_dequant_linear_workspace_bytes(L.QB_BF16, M, K, N) + 16, dtype=torch.uint8, device=DEV)
    wb = torch.empty(L.qb_dequant_linear_backward_workspace_bytes(L.QB_BF16, M, K, N), dtype=torch.uint8, device=DEV)
    dq = w.dq(L)

    def step():
        L.qb_dequant_linear(x, w.codes, None, NF4, 64, N, y, ws, bias=bias, act=L.QB_ACT_GELU, z=z, dq=dq)
        L.qb_dequant_linear_backward(dy, w.codes, None, NF4, 64, K, dx, wb, act=L.QB_ACT_GELU, z=z, dbias=db, dq=dq)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(ref.normal((M, K), 10 + i, dtype=BF16))
        dy.copy_(ref.normal((M, N), 20 + i, dtype=BF16))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (y, z, dx, db)]
        for t in (y, z, dx, db):
            t.fill_(9.0)
        ws.fill_(0xEE)
        wb.fill_(0xEE)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, z, dx, db), want))


def test_streams_and_repeats():
    """The same bits on another stream, and again; two calls at once with workspaces of their own."""
    L = qb()
    w = ref.Weight(260, 512, NF4, 64, False, F16, seed=5)
    xs = [ref.normal((140, 512), i, dtype=F16) for i in range(2)]
    want = [forward(L, x, w, act="GELU") for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    size = L.qb_dequant_linear_workspace_bytes(L.QB_F16, 140, 512, 260)
    wss = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in xs]
    ys = [torch.empty(140, 260, dtype=F16, device=DEV) for _ in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        for x, y, ws, s in zip(xs, ys, wss, streams):
            L.qb_dequant_linear(x, w.codes, w.absmax, NF4, 64, 260, y, ws, act=L.QB_ACT_GELU, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ys, want))


def test_binding_refuses_wrong_shapes_and_types():
    L = qb()
    w = ref.Weight(64, 128, NF4, 64, True, BF16, seed=1)
    x, y = ref.normal((4, 128), 1, dtype=BF16), torch.empty(4, 64, dtype=BF16, device=DEV)
    call = lambda **kw: L.qb_dequant_linear(**{**dict(x=x, codes=w.codes, absmax=None, code=NF4, blocksize=64, N=64,  # noqa: E731
                                                      y=y, dq=w.dq(L)), **kw})
    call()
    for bad in (dict(y=y[:3]), dict(y=y.float()), dict(codes=w.codes[:-1]), dict(codes=w.codes.view(torch.int8)),
                dict(residual=y[:, :32]), dict(z=y.float()), dict(bias=torch.empty(63, device=DEV)),
                dict(dq=L.make_dq(w.dq_parts[0][:-1], *w.dq_parts[1:], 256)), dict(x=x.t()), dict(x=x.cpu()),
                dict(bias=torch.empty(64))):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    for status, bad in ((L.QB_EUNSUPPORTED, dict(bias=torch.empty(64, dtype=F16, device=DEV))),
                        (L.QB_EINVAL, dict(act=5)), (L.QB_EINVAL, dict(code=L.QB_DYN8)), (L.QB_EINVAL, dict(blocksize=96))):
        with pytest.raises(L.QbError) as e:
            call(**bad)
        assert e.value.status == status
    with pytest.raises(L.QbError) as e:                 # 65 rows need a workspace
        L.qb_dequant_linear(ref.normal((65, 128), 1, dtype=BF16), w.codes, None, NF4, 64, 64,
                            torch.empty(65, 64, dtype=BF16, device=DEV), dq=w.dq(L))
    assert e.value.status == L.QB_EINVAL


# products of enough tiles for the larger tile shapes, ragged at both ends: 256 x 256 (15 x 14 forward, 15 x 14
# backward), 128 x 128 (12 x 17)
LARGE = [(3600, 160, 3501), (3601, 3520, 130), (1500, 224, 2111), (1499, 2112, 97)]


@pytest.mark.parametrize("M,K,N", LARGE)
@pytest.mark.parametrize("xdt", [BF16, F16, F32])
def test_large_tiles(M, K, N, xdt):
    L = qb()
    w = ref.Weight(N, K, NF4, 64, True, xdt, seed=M)
    x, bias, residual = (ref.normal(s, M + i, dtype=xdt) for i, s in enumerate([(M, K), (N,), (M, N)]))
    y, z = forward(L, x, w, bias, "GELU", residual, keep=True)
    check_forward(L, x, w, bias, "GELU", residual, y, z)
    assert torch.equal(forward(L, x, w, bias, "GELU", residual, in_place=True), y)
    dy = ref.normal((M, N), 5, 0.1, xdt)
    dx, dz, db = backward(L, dy, w, z, "GELU", dz=True, bias_dt=F32)
    check_backward(L, dy, w, z, "GELU", dx, dz, db)
