"""GPU: the gated block of two 4-bit weights and its gradient against the binary64
formulas within the rounding error of their evaluation (linear_reference.py)."""
import numpy as np
import pytest
import torch

import linear_reference as ref
import oracle
from gpu_helpers import DEV, qb
from test_gpu_linear import ACTS, BF16, F16, F32, kind_of, workspace

pytestmark = pytest.mark.gpu

NF4, FP4 = oracle.NF4, oracle.FP4


def pair(n, k, code, blocksize, nested, xdt, seed, blocksize2=256):
    return [ref.Weight(n, k, code, blocksize, nested, xdt, seed + i, blocksize2) for i in range(2)]


def forward(L, x, w, act="SILU", keep=False):
    m, n = x.shape[0], w[0].n
    ws, guard = workspace(L.qb_dequant_gated_workspace_bytes(L._DTYPE[x.dtype], m, w[0].k, n))
    y, g, u = (torch.full((m + 1, n), 7.0, dtype=x.dtype, device=DEV) for _ in range(3))
    L.qb_dequant_gated(x, w[0].parts(L), w[1].parts(L), w[0].code, w[0].blocksize, n, y[:m], ws, act=kind_of(L, act),
                       gate_out=g[:m] if keep else None, up_out=u[:m] if keep else None)
    torch.cuda.synchronize()
    assert (guard == 0x5A).all() and all((t[m:] == 7.0).all() for t in (y, g, u))
    return (y[:m], g[:m], u[:m]) if keep else y[:m]


def backward(L, dy, g, u, w, act="SILU", dx=True, keep=(False, False)):
    m, n = dy.shape
    ws, guard = workspace(L.qb_dequant_gated_backward_workspace_bytes(L._DTYPE[dy.dtype], m, w[0].k, n))
    gx = torch.full((m + 1, w[0].k), 7.0, dtype=dy.dtype, device=DEV)
    outs = [torch.full((m + 1, n), 7.0, dtype=dy.dtype, device=DEV) for _ in range(2)]
    L.qb_dequant_gated_backward(dy, g, u, w[0].parts(L), w[1].parts(L), w[0].code, w[0].blocksize, w[0].k,
                                gx[:m] if dx else None, ws, act=kind_of(L, act), dgate=outs[0][:m] if keep[0] else None,
                                dup=outs[1][:m] if keep[1] else None)
    torch.cuda.synchronize()
    assert (guard == 0x5A).all() and (gx[m if dx else 0:] == 7.0).all()
    assert all((t[m if k else 0:] == 7.0).all() for t, k in zip(outs, keep))
    return (gx[:m] if dx else None, *(t[:m] if k else None for t, k in zip(outs, keep)))


def check_forward(L, x, w, act, y, g=None, u=None):
    want_g, eg, want_u, eu, want, e = ref.gated(L, ref.f64(x), w[0].w, w[1].w, kind_of(L, act))
    ref.assert_close(y, want, e, "y")
    if g is not None:
        ref.assert_close(g, want_g, eg, "gate")
    if u is not None:
        ref.assert_close(u, want_u, eu, "up")


def check_backward(L, dy, g, u, w, act, dx, dg=None, du=None):
    d, uv = ref.f64(dy), ref.f64(u)
    a, slope, ea, es = ref.act(L, kind_of(L, act), ref.f64(g))
    want_g, want_u = d * uv * slope, d * a
    eg = np.abs(d * uv) * es + 2 * ref.U * np.abs(want_g)
    eu = np.abs(d) * ea + ref.U * np.abs(want_u)
    if dg is not None:
        ref.assert_close(dg, want_g, eg, "dgate")
    if du is not None:
        ref.assert_close(du, want_u, eu, "dup")
    if dx is not None:
        both = np.concatenate([want_g, want_u], 1), np.concatenate([eg, eu], 1), np.concatenate([w[0].w, w[1].w], 0)
        ref.assert_close(dx, *ref.rounded_product(*both, dy.dtype), "dx")


SHAPES = [(1, 4096, 300), (8, 512, 64), (9, 160, 40), (16, 32, 3), (17, 1024, 40), (33, 96, 17), (64, 256, 48),
          (65, 256, 48), (65, 32, 1), (100, 96, 131), (128, 64, 128), (129, 1056, 130), (200, 992, 1001), (300, 128, 4)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("xdt", [BF16, F16, F32])
def test_shapes_and_types(M, K, N, xdt):
    L = qb()
    print(f"[gated] {M} {K} {N} {xdt}", flush=True)
    w = pair(N, K, NF4, 64, False, xdt, seed=M + K + N)
    x = ref.normal((M, K), M, 1.0 / np.sqrt(K) * 10, dtype=xdt)
    y, g, u = forward(L, x, w, keep=True)
    check_forward(L, x, w, "SILU", y, g, u)
    assert torch.equal(forward(L, x, w), y)
    dy = ref.normal((M, N), 5, 0.1, xdt)
    dx, dg, du = backward(L, dy, g, u, w, keep=(True, True))
    check_backward(L, dy, g, u, w, "SILU", dx, dg, du)
    for keep in ((False, False), (True, False), (False, True)):
        other = backward(L, dy, g, u, w, keep=keep)
        assert torch.equal(other[0], dx)
        assert other[1] is None or torch.equal(other[1], dg)
        assert other[2] is None or torch.equal(other[2], du)
    assert torch.equal(backward(L, dy, g, u, w, dx=False, keep=(True, True))[1], dg)


@pytest.mark.parametrize("M", [7, 40, 150])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("xdt", [BF16, F32])
def test_activations(M, act, xdt):
    L = qb()
    w = pair(73, 128, FP4, 128, False, xdt, seed=3)
    x = ref.normal((M, 128), 1, 2.0, xdt)
    y, g, u = forward(L, x, w, act, keep=True)
    check_forward(L, x, w, act, y, g, u)
    dy = ref.normal((M, 73), 4, 1.0, xdt)
    check_backward(L, dy, g, u, w, act, *backward(L, dy, g, u, w, act, keep=(True, True)))


@pytest.mark.parametrize("code", [NF4, FP4])
@pytest.mark.parametrize("blocksize,blocksize2", [(64, 256), (512, 64), (4096, 4096)])
@pytest.mark.parametrize("nested", [False, True])
@pytest.mark.parametrize("M", [5, 40, 90])
def test_codes_blocks_and_nesting(code, blocksize, blocksize2, nested, M):
    L = qb()
    w = pair(200, 1120, code, blocksize, nested, BF16, blocksize + code, blocksize2)
    x = ref.normal((M, 1120), 1, 0.3, dtype=BF16)
    y, g, u = forward(L, x, w, "GELU", keep=True)
    check_forward(L, x, w, "GELU", y, g, u)
    dy = ref.normal((M, 200), 2, dtype=BF16)
    check_backward(L, dy, g, u, w, "GELU", backward(L, dy, g, u, w, "GELU")[0])


@pytest.mark.parametrize("M", [30, 70, 300])
@pytest.mark.parametrize("xdt", [BF16, F32])
def test_every_weight_in_its_place(M, xdt):
    """Rows of the identity give back both weights bit for bit; in the other direction relu with gate and up of
    ones and zeros takes the rows of one of them."""
    L = qb()
    for n, k in ((137, 160), (320, 96)):
        w = pair(n, k, NF4, 64, True, xdt, seed=n)
        values = [v.values.to(DEV) for v in w]
        for at in range(0, max(n, k), M):
            rows = torch.arange(at, at + M, device=DEV)
            x = torch.zeros(M, k, dtype=xdt, device=DEV)
            live = rows < k
            x[live, rows[live]] = 1.0
            _, g, u = forward(L, x, w, keep=True)
            for got, v in ((g, values[0]), (u, values[1])):
                want = torch.zeros(M, n, dtype=xdt, device=DEV)
                want[live] = v[:, rows[live]].T
                assert torch.equal(got, want)
            dy = torch.zeros(M, n, dtype=xdt, device=DEV)
            live = rows < n
            dy[live, rows[live]] = 1.0
            one, zero = torch.ones_like(dy), torch.zeros_like(dy)
            for g, u, v in ((one, one * 0, values[1]), (zero, one, None), (one * 0.5, one, values)):
                dx = backward(L, dy, g.contiguous(), u.contiguous(), w, "RELU")[0]
                want = torch.zeros(M, k, dtype=xdt, device=DEV)
                if v is values:                          # dg = dy, du = dy / 2: two terms, rounded once
                    want[live] = (values[0].double()[rows[live]] + values[1].double()[rows[live]] / 2).to(xdt)
                elif v is not None:
                    want[live] = v[rows[live]]
                assert torch.equal(dx, want)


@pytest.mark.parametrize("M", [6, 130])
def test_captured_calls_replay(M):
    L = qb()
    K, N = 256, 200
    w = pair(N, K, NF4, 64, True, BF16, seed=4)
    x, dy = ref.normal((M, K), 1, dtype=BF16), ref.normal((M, N), 2, dtype=BF16)
    y, g, u, dx = (torch.empty(M, n, dtype=BF16, device=DEV) for n in (N, N, N, K))
    ws = torch.empty(L.qb_dequant_gated_workspace_bytes(L.QB_BF16, M, K, N) + 16, dtype=torch.uint8, device=DEV)
    wb = torch.empty(L.qb_dequant_gated_backward_workspace_bytes(L.QB_BF16, M, K, N), dtype=torch.uint8, device=DEV)
    parts = [v.parts(L) for v in w]

    def step():
        L.qb_dequant_gated(x, *parts, NF4, 64, N, y, ws, gate_out=g, up_out=u)
        L.qb_dequant_gated_backward(dy, g, u, *parts, NF4, 64, K, dx, wb)

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
        want = [t.clone() for t in (y, g, u, dx)]
        for t in (y, g, u, dx):
            t.fill_(9.0)
        ws.fill_(0xEE)
        wb.fill_(0xEE)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, g, u, dx), want))


@pytest.mark.parametrize("M", [20, 100])
def test_nan_stays_in_its_row(M):
    L = qb()
    w = pair(80, 96, NF4, 64, False, BF16, seed=1)
    x = ref.normal((M, 96), 1, dtype=BF16)
    clean, g, u = forward(L, x, w, keep=True)
    x[3, 95] = float("nan")
    y = forward(L, x, w)
    rows = torch.ones(M, dtype=torch.bool)
    rows[3] = False
    assert torch.equal(y[rows], clean[rows]) and y[3].isnan().all()
    dy = ref.normal((M, 80), 2, dtype=BF16)
    clean = backward(L, dy, g, u, w)[0]
    dy[3, 79] = float("nan")
    dx = backward(L, dy, g, u, w)[0]
    assert torch.equal(dx[rows], clean[rows]) and dx[3].isnan().all()


def test_no_rows_and_refusals():
    L = qb()
    w = pair(64, 128, NF4, 64, True, BF16, seed=1)
    empty = torch.empty(0, 64, dtype=BF16, device=DEV)
    forward(L, torch.empty(0, 128, dtype=BF16, device=DEV), w)
    backward(L, empty, empty, empty, w)
    x, y = ref.normal((4, 128), 1, dtype=BF16), torch.empty(4, 64, dtype=BF16, device=DEV)
    plain = ref.Weight(64, 128, NF4, 64, False, BF16, seed=1)
    call = lambda **kw: L.qb_dequant_gated(**{**dict(x=x, gate=w[0].parts(L), up=w[1].parts(L), code=NF4, blocksize=64,  # noqa: E731
                                                     N=64, y=y), **kw})
    call()
    other = (w[1].codes, None, L.make_dq(*w[1].dq_parts, 64))
    for bad in (dict(y=y[:3]), dict(gate_out=y.float()), dict(up=(w[1].codes[:-1], None, w[1].dq(L))), dict(up=other),
                dict(x=x.t()), dict(x=x.cpu())):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    for status, bad in ((L.QB_EUNSUPPORTED, dict(up=plain.parts(L))), (L.QB_EINVAL, dict(act=-1)),
                        (L.QB_EINVAL, dict(gate=(w[0].codes, None, None)))):
        with pytest.raises(L.QbError) as e:
            call(**bad)
        assert e.value.status == status


@pytest.mark.parametrize("M,K,N", [(3600, 160, 1751), (3601, 3520, 67), (1500, 224, 1055), (1499, 2112, 49)])
@pytest.mark.parametrize("xdt", [BF16, F16, F32])
def test_large_tiles(M, K, N, xdt):
    L = qb()
    w = pair(N, K, NF4, 64, True, xdt, seed=M)
    x = ref.normal((M, K), M, 10 / np.sqrt(K), dtype=xdt)
    y, g, u = forward(L, x, w, keep=True)
    check_forward(L, x, w, "SILU", y, g, u)
    dy = ref.normal((M, N), 5, 0.1, xdt)
    dx, dg, du = backward(L, dy, g, u, w, keep=(True, True))
    check_backward(L, dy, g, u, w, "SILU", dx, dg, du)
