"""GPU: the forward pass of the 4-bit layers through the dequantized weights and the tiled product, which
calls of more than 1024 rows take whatever the estimates say (inputs of 64 at least): every type, code, block size, nesting
and activation against the binary64 formulas within the rounding error of their evaluation
(linear_reference.py).  Every call here must have left the weights, bit for bit, in its workspace."""
import pytest
import torch

import linear_reference as ref
import oracle
import test_gpu_gated as gated
import test_gpu_linear as linear
from gpu_helpers import DEV, qb
from test_gpu_linear import ACTS, BF16, F16, F32, kind_of

pytestmark = pytest.mark.gpu

NF4, FP4 = oracle.NF4, oracle.FP4
M = 1030



AT = [0, 1, 63, 64, 127, 128, 255, 256, 511, 512, 700, 1023, 1024, 1025, M - 2, M - 1]


def in_workspace(ws, weights, xdt):
    """The weights in the compute dtype at the workspace's beginning, each at a multiple of 256 bytes."""
    at = 0
    for w in weights:
        size = w.n * w.k * (4 if xdt == F32 else 2)
        kept = ws[at:at + size].view(xdt).view(w.n, w.k)
        assert torch.equal(kept, w.values.to(DEV)), "not the tiled product"
        at += -(-size // 256) * 256


def forward(L, x, w, bias=None, act="NONE", residual=None, keep=False, in_place=False):
    """As linear.forward, the weights looked for in the workspace."""
    m, n = x.shape[0], w.n
    ws, guard = linear.workspace(L.qb_dequant_linear_workspace_bytes(L._DTYPE[x.dtype], m, w.k, n))
    y = torch.full((m + 1, n), 7.0, dtype=x.dtype, device=DEV)
    z = torch.full((m + 1, n), 7.0, dtype=x.dtype, device=DEV) if keep else None
    if in_place:
        y[:m] = residual
        residual = y[:m]
    L.qb_dequant_linear(x, w.codes, w.absmax, w.code, w.blocksize, n, y[:m], ws, bias=bias, act=kind_of(L, act),
                        residual=residual, z=z[:m] if keep else None, dq=w.dq(L))
    torch.cuda.synchronize()
    assert (guard == 0x5A).all() and (y[m:] == 7.0).all() and (z is None or (z[m:] == 7.0).all())
    in_workspace(ws, [w], x.dtype)
    return (y[:m], z[:m]) if keep else y[:m]


def forward_gated(L, x, w, act="SILU"):
    m, n = x.shape[0], w[0].n
    ws, guard = linear.workspace(L.qb_dequant_gated_workspace_bytes(L._DTYPE[x.dtype], m, w[0].k, n))
    y, g, u = (torch.full((m + 1, n), 7.0, dtype=x.dtype, device=DEV) for _ in range(3))
    L.qb_dequant_gated(x, w[0].parts(L), w[1].parts(L), w[0].code, w[0].blocksize, n, y[:m], ws, act=kind_of(L, act),
                       gate_out=g[:m], up_out=u[:m])
    torch.cuda.synchronize()
    assert (guard == 0x5A).all() and all((t[m:] == 7.0).all() for t in (y, g, u))
    in_workspace(ws, w, x.dtype)
    return y[:m], g[:m], u[:m]


def check_linear(L, x, w, bias, act, residual, y, z=None, at=AT):
    at = torch.tensor(at, device=DEV)
    linear.check_forward(L, x[at], w, bias, act, None if residual is None else residual[at], y[at],
                         None if z is None else z[at])


def check_gated(L, x, w, act, y, g, u, at=AT):
    at = torch.tensor(at, device=DEV)
    gated.check_forward(L, x[at], w, act, y[at], g[at], u[at])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("xdt", [BF16, F16, F32])
@pytest.mark.parametrize("K,N", [(128, 73), (96, 300), (1056, 65)])
def test_activations(act, xdt, K, N):
    """Steps of the whole length and a last half one; outputs in whole groups of eight and beyond them."""
    L = qb()
    w = gated.pair(N, K, FP4, 128, False, xdt, 3)
    x = ref.normal((M, K), 1, 20 / K ** 0.5, xdt)
    bias, residual = ref.normal((N,), 2, 3.0), ref.normal((M, N), 4, dtype=xdt)
    y, z = forward(L, x, w[0], bias, act, residual, keep=True)
    check_linear(L, x, w[0], bias, act, residual, y, z)
    check_gated(L, x, w, act, *forward_gated(L, x, w, act))


@pytest.mark.parametrize("code", [NF4, FP4])
@pytest.mark.parametrize("blocksize,blocksize2", [(64, 256), (128, 64), (256, 4096), (512, 256), (1024, 128),
                                                  (2048, 512), (4096, 1024)])
@pytest.mark.parametrize("nested", [False, True])
@pytest.mark.parametrize("xdt", [BF16, F16, F32])
def test_codes_blocks_and_nesting(code, blocksize, blocksize2, nested, xdt):
    L = qb()
    w = gated.pair(117, 1120, code, blocksize, nested, xdt, blocksize + code, blocksize2)
    x = ref.normal((M, 1120), 1, 0.3, dtype=xdt)
    check_linear(L, x, w[0], None, "NONE", None, forward(L, x, w[0]))
    check_gated(L, x, w, "GELU", *forward_gated(L, x, w, "GELU"))


@pytest.mark.parametrize("xdt", [BF16, F16, F32])
def test_every_weight_in_its_place(xdt):
    """Rows of the identity give back the weights bit for bit."""
    L = qb()
    for n, k in ((137, 160), (320, 96), (70, 1024)):
        w = gated.pair(n, k, NF4, 64, True, xdt, n)
        x = torch.zeros(M, k, dtype=xdt, device=DEV)
        x[3:3 + k] = torch.eye(k, dtype=xdt, device=DEV)
        _, g, u = forward_gated(L, x, w)
        for got, v in ((forward(L, x, w[0]), w[0]), (g, w[0]), (u, w[1])):
            want = torch.zeros(M, n, dtype=xdt, device=DEV)
            want[3:3 + k] = v.values.to(DEV).T
            assert torch.equal(got, want)


@pytest.mark.parametrize("N", [64, 129])
@pytest.mark.parametrize("xdt", [BF16, F32])
def test_parts_of_the_epilogue(N, xdt):
    """Each optional input and output with and without the others; the residual in place."""
    L = qb()
    w = ref.Weight(N, 256, NF4, 64, True, xdt, seed=1)
    x, residual = ref.normal((M, 256), 0, dtype=xdt), ref.normal((M, N), 1, dtype=xdt)
    for bias in (None, ref.normal((N,), 7), ref.normal((N,), 8, dtype=xdt)):
        for res in (None, residual):
            for act in ("NONE", "GELU_TANH"):
                y, z = forward(L, x, w, bias, act, res, keep=True)
                check_linear(L, x, w, bias, act, res, y, z)
                assert torch.equal(forward(L, x, w, bias, act, res), y)
                if res is not None:
                    assert torch.equal(forward(L, x, w, bias, act, res, in_place=True), y)


@pytest.mark.parametrize("xdt", [BF16, F16, F32])
def test_infinities_and_nan_stay_in_their_rows(xdt):
    L = qb()
    w = gated.pair(80, 96, NF4, 64, False, xdt, 1)
    x = ref.normal((M, 96), 1, dtype=xdt)
    clean, clean_gated = forward(L, x, w[0]), forward_gated(L, x, w)
    bad = [3, 255, 700, M - 1]
    x[3, 95], x[255, 0], x[700, 64], x[M - 1, 5] = float("nan"), float("nan"), float("nan"), float("inf")
    rows = torch.ones(M, dtype=torch.bool, device=DEV)
    rows[bad] = False
    y = forward(L, x, w[0])
    assert torch.equal(y[rows], clean[rows]) and y[bad[:3]].isnan().all()
    assert y[M - 1][(w[0].values[:, 5] != 0).to(DEV)].isinf().all()
    for got, c in zip(forward_gated(L, x, w), clean_gated):
        assert torch.equal(got[rows], c[rows]) and got[bad[:3]].isnan().all()


@pytest.mark.parametrize("xdt", [BF16, F16])
def test_captured_calls_replay(xdt):
    """Linear, gated and both gradients in one graph on one workspace, replayed on new inputs with eager work in
    between and the workspace overwritten."""
    L = qb()
    K, N = 160, 200
    w, dt = gated.pair(N, K, NF4, 64, True, xdt, 4), L._DTYPE[xdt]
    x, dy, bias = ref.normal((M, K), 1, dtype=xdt), ref.normal((M, N), 2, dtype=xdt), ref.normal((N,), 3)
    y, z, h, g, u, dx, dx2 = (torch.empty(M, n, dtype=xdt, device=DEV) for n in (N, N, N, N, N, K, K))
    db = torch.empty(N, device=DEV)
    ws = torch.empty(max(f(dt, M, K, N) for f in (
        L.qb_dequant_linear_workspace_bytes, L.qb_dequant_linear_backward_workspace_bytes,
        L.qb_dequant_gated_workspace_bytes, L.qb_dequant_gated_backward_workspace_bytes)), dtype=torch.uint8, device=DEV)
    parts = [v.parts(L) for v in w]

    def step():
        L.qb_dequant_linear(x, w[0].codes, None, NF4, 64, N, y, ws, bias=bias, act=L.QB_ACT_GELU, z=z, dq=parts[0][2])
        L.qb_dequant_linear_backward(dy, w[0].codes, None, NF4, 64, K, dx, ws, act=L.QB_ACT_GELU, z=z, dbias=db,
                                     dq=parts[0][2])
        L.qb_dequant_gated(x, *parts, NF4, 64, N, h, ws, gate_out=g, up_out=u)
        L.qb_dequant_gated_backward(dy, g, u, *parts, NF4, 64, K, dx2, ws)

    outs = (y, z, h, g, u, dx, dx2, db)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(ref.normal((M, K), 10 + i, dtype=xdt))
        dy.copy_(ref.normal((M, N), 20 + i, dtype=xdt))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(9.0)
        ws.fill_(0xEE)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("xdt", [BF16, F32])
def test_two_calls_at_once(xdt):
    """Two streams, a workspace each, other weights: the bits of the same calls one after the other."""
    L = qb()
    K, N = 512, 260
    ws_ = [ref.Weight(N, K, NF4, 64, False, xdt, seed=5 + i) for i in range(2)]
    xs = [ref.normal((M, K), i, dtype=xdt) for i in range(2)]
    want = [forward(L, x, w, act="GELU") for x, w in zip(xs, ws_)]
    streams = [torch.cuda.Stream() for _ in xs]
    size = L.qb_dequant_linear_workspace_bytes(L._DTYPE[xdt], M, K, N)
    wss = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in xs]
    ys = [torch.empty(M, N, dtype=xdt, device=DEV) for _ in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        for x, w, y, ws, s in zip(xs, ws_, ys, wss, streams):
            L.qb_dequant_linear(x, w.codes, w.absmax, NF4, 64, N, y, ws, act=L.QB_ACT_GELU, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ys, want))
    for ws, w in zip(wss, ws_):
        in_workspace(ws, [w], xdt)


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 6, 7])
@pytest.mark.parametrize("rows", [3, 65, 130])
@pytest.mark.parametrize("xdt", [BF16, F16, F32])
def test_nested_weights_of_few_outputs(N, rows, xdt):
    """Gradients through nested weights whose rows of dz are shorter than a unit of eight."""
    L = qb()
    K = 352
    w = gated.pair(N, K, NF4, 64, True, xdt, N, 64)
    dy, z, u = (ref.normal((rows, N), i, 0.5, xdt) for i in range(3))
    dx, dz, db = linear.backward(L, dy, w[0], z, "SILU", dz=True, bias_dt=F32)
    linear.check_backward(L, dy, w[0], z, "SILU", dx, dz, db)
    linear.check_backward(L, dy, w[0], None, "NONE", linear.backward(L, dy, w[0])[0], None, None)
    gated.check_backward(L, dy, z, u, w, "GELU", *gated.backward(L, dy, z, u, w, "GELU", keep=(True, True)))
