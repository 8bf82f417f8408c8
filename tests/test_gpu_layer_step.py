"""GPU: the 4-bit layers, their gradients and the clipping as a training step uses them, with the
framework's embedding, layer norm and optimizer around them: every stage against its formula in
64 bits on the inputs that it had, the chain's gradient against autograd in 64 bits, the step
captured and replayed; then the layers fed one token, or a few, at a time."""
import pytest
import torch

import linear_reference as ref
import oracle
import test_gpu_gated as gated
import test_gpu_grad_norm as clip
import test_gpu_layer_norm as norm
import test_gpu_linear as linear
from gpu_helpers import DEV, qb

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ROWS, DIM, WIDE, EPS = 90, 160, 352, 1e-5


class Block:
    """ids -> embedding -> layer norm -> gated block -> 4-bit layer with bias, plus the embedding."""

    def __init__(self, L, tokens, xdt, nested=True):
        self.L, self.tokens, self.xdt = L, tokens, xdt
        self.gate, self.up = gated.pair(WIDE, DIM, oracle.NF4, 64, nested, xdt, 1)
        self.down = ref.Weight(DIM, WIDE, oracle.NF4, 64, nested, xdt, 3)
        self.table = ref.normal((ROWS, DIM), 4, 1.0, xdt)
        self.gamma = 1 + ref.normal((DIM,), 5, 0.2, xdt)
        self.beta, self.bias = ref.normal((DIM,), 6, 0.2, xdt), ref.normal((DIM,), 7, 0.2, xdt)
        self.params = [self.table, self.gamma, self.beta, self.bias]
        self.grads = [torch.empty_like(p) for p in self.params]
        self.ids = torch.randint(0, ROWS, (tokens,), device=DEV)
        self.target = ref.normal((tokens, DIM), 8, 1.0, xdt)
        new = lambda width, dt=xdt: torch.empty(tokens, width, dtype=dt, device=DEV)  # noqa: E731
        self.x, self.h, self.y, self.dy, self.dh, self.dx = (new(DIM) for _ in range(6))
        self.g, self.u, self.a, self.da = (new(WIDE) for _ in range(4))
        self.mean, self.rstd = (torch.empty(tokens, device=DEV) for _ in range(2))
        dt, byte = L._DTYPE[xdt], torch.uint8
        self.ws = torch.empty(max(L.qb_dequant_gated_workspace_bytes(dt, tokens, DIM, WIDE),
                                  L.qb_dequant_linear_workspace_bytes(dt, tokens, WIDE, DIM),
                                  L.qb_dequant_linear_backward_workspace_bytes(dt, tokens, WIDE, DIM),
                                  L.qb_dequant_gated_backward_workspace_bytes(dt, tokens, DIM, WIDE),
                                  L.qb_layer_norm_workspace_bytes(tokens, DIM),
                                  L.qb_embedding_workspace_bytes(tokens, ROWS, DIM),
                                  L.qb_multi_tensor_grad_norm_workspace_bytes(4)), dtype=byte, device=DEV)
        self.weights = [w.parts(L) for w in (self.gate, self.up, self.down)]
        self.grad_table, self.norm = L.grad_table(self.grads), torch.empty(1, device=DEV)
        from bit_optimizer_states_amd import state
        self.states = state.allocate(self.params, L.QB_ADAMW, blocksize=256, force_32bit=(1, 2, 3))
        self.tensors = L.tensor_table([(p, g, *s[:4]) for p, g, s in zip(self.params, self.grads, self.states)])
        self.hp = L.optim_hparams(L.QB_ADAMW, 1e-2, 0.9, 0.999, 1e-8, 0.01, step=1)
        self.opt_ws = torch.empty(L.qb_optimizer_workspace_bytes(self.hp, self.tensors, 4, 256), dtype=byte, device=DEV)

    def forward(self):
        L = self.L
        L.qb_embedding(self.table, self.ids, self.x)
        L.qb_layer_norm(self.x, self.gamma, self.beta, EPS, self.h, self.mean, self.rstd)
        gate, up, (codes, absmax, dq) = self.weights
        L.qb_dequant_gated(self.h, gate, up, oracle.NF4, 64, WIDE, self.a, self.ws, gate_out=self.g, up_out=self.u)
        L.qb_dequant_linear(self.a, codes, absmax, oracle.NF4, 64, DIM, self.y, self.ws, bias=self.bias,
                            residual=self.x, dq=dq)

    def backward(self):
        """Of half the squared error over the tokens."""
        L = self.L
        torch.sub(self.y, self.target, out=self.dy)
        self.dy.mul_(1.0 / self.tokens)
        gate, up, (codes, absmax, dq) = self.weights
        L.qb_dequant_linear_backward(self.dy, codes, absmax, oracle.NF4, 64, WIDE, self.da, self.ws,
                                     dbias=self.grads[3], dq=dq)
        L.qb_dequant_gated_backward(self.da, self.g, self.u, gate, up, oracle.NF4, 64, DIM, self.dh, self.ws)
        L.qb_layer_norm_backward(self.dh, self.x, self.gamma, self.mean, self.rstd, self.dx, self.grads[1],
                                 self.grads[2], self.ws)
        self.dx.add_(self.dy)
        L.qb_embedding_backward(self.dx, self.ids, self.grads[0], self.ws)

    def clip(self, max_norm):
        self.L.qb_multi_tensor_grad_norm(self.grad_table, 4, self.norm, self.ws)
        self.L.qb_multi_tensor_clip_grads(self.grad_table, 4, max_norm, self.norm)

    def optimizer(self):
        dt = self.L._DTYPE[self.xdt]
        self.L.qb_multi_tensor_optimizer_step(self.hp, self.tensors, 4, dt, 256, self.opt_ws, pdt=dt)

    def gradients(self):
        self.forward()
        self.backward()
        self.clip(0.5)

    def step(self):
        self.gradients()
        self.optimizer()

    def results(self):
        return [self.y, self.dx, self.norm, *self.grads, *self.params, *(t for s in self.states for t in s[:4] if t is not None)]


@pytest.mark.parametrize("tokens", [1, 40, 200])
@pytest.mark.parametrize("xdt", [BF16, F32])
def test_every_stage_of_three_steps(tokens, xdt):
    L = qb()
    b = Block(L, tokens, xdt)
    for step in (1, 2, 3):
        print(f"[step] {tokens} {xdt} {step}", flush=True)
        b.hp.step = step
        b.ids.copy_(torch.randint(0, ROWS, (tokens,), device=DEV))
        b.forward()
        b.backward()
        torch.cuda.synchronize()
        assert torch.equal(b.x, b.table[b.ids])
        norm.check_forward(b.x, b.gamma, b.beta, b.h, b.mean, b.rstd, EPS)
        w = (b.gate, b.up)
        gated.check_forward(L, b.h, w, "SILU", b.a, b.g, b.u)
        linear.check_forward(L, b.a, b.down, b.bias, "NONE", b.x, b.y)
        linear.check_backward(L, b.dy, b.down, None, "NONE", b.da, None, b.grads[3])
        gated.check_backward(L, b.da, b.g, b.u, w, "SILU", b.dh)
        norm.check_backward(b.x, b.gamma, b.dh, b.mean, b.rstd, None, b.grads[1], b.grads[2])
        before = [g.clone() for g in b.grads]
        b.clip(0.5)
        torch.cuda.synchronize()
        want = clip.exact_norm(before)
        assert abs(b.norm.item() - want) <= want * 2.0 ** -24 * 1.001 and want > 0.5
        for g, old in zip(b.grads, before):
            assert torch.equal(g, clip.expected(old, 0.5, b.norm))
        old = [p.clone() for p in b.params]
        b.optimizer()
        torch.cuda.synchronize()
        assert all(p.isfinite().all() and not torch.equal(p, o) for p, o in zip(b.params, old))


@pytest.mark.parametrize("tokens", [40, 200])
def test_chain_against_autograd_in_64_bits(tokens):
    """The gradients of the whole block in binary32.  Seven stages, each off by at most (k + 2) 2u of its sum of
    absolute terms, k <= 352, i.e. 4.3e-5 of it; these sums stay within 16 of the largest value for random
    signs (sqrt(352) = 19 at the typical one), so 7 * 16 * 4.3e-5 = 2^-7.7 of the largest gradient at the worst."""
    L = qb()
    b = Block(L, tokens, F32)
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    leaves = [p.cpu().double().requires_grad_() for p in b.params]
    table, gamma, beta, bias = leaves
    x = table[b.ids.cpu()]
    h = torch.nn.functional.layer_norm(x, (DIM,), gamma, beta, EPS)
    wg, wu, wd = (w.values.double() for w in (b.gate, b.up, b.down))
    y = (torch.nn.functional.silu(h @ wg.T) * (h @ wu.T)) @ wd.T + bias + x
    ((y - b.target.cpu().double()) ** 2).sum().div(2 * tokens).backward()
    for got, leaf in zip(b.grads, leaves):
        assert (got.cpu().double() - leaf.grad).abs().max() <= 2.0 ** -7.7 * leaf.grad.abs().max()


@pytest.mark.parametrize("tokens", [40, 200])
@pytest.mark.parametrize("xdt", [BF16, F32])
def test_captured_step_replays(tokens, xdt):
    """Forward, backward and clipping in one graph, one workspace shared by all its calls, against the eager step
    from the same state; two graphs in turn.  The optimizer's call stays outside: it uploads its table of tensors
    from host memory that the next call's table replaces."""
    L = qb()
    blocks = [Block(L, tokens, xdt), Block(L, tokens + 30, xdt, nested=False)]
    graphs = []
    for b in blocks:
        b.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.gradients()
        graphs.append(g)
    for turn in range(4):
        wants, starts = [], []
        for b in blocks:
            b.ids.copy_(torch.randint(0, ROWS, b.ids.shape, device=DEV))
            starts.append([t.clone() for t in b.results()])
            b.step()
            torch.cuda.synchronize()
            wants.append([t.clone() for t in b.results()])
        for b, start in zip(blocks, starts):
            for t, s in zip(b.results(), start):
                t.copy_(s)
            b.ws.fill_(0xEE)
        for b, g in zip(blocks, graphs):
            g.replay()
            b.optimizer()
        torch.cuda.synchronize()
        for b, want in zip(blocks, wants):
            assert all(torch.equal(t, w) for t, w in zip(b.results(), want)), turn


def test_two_steps_at_once_on_streams():
    """Two blocks on streams of their own, a workspace each, equal the same steps one after the other."""
    L = qb()
    blocks = [Block(L, 130, BF16), Block(L, 50, BF16)]
    starts = [[t.clone() for t in b.results()] for b in blocks]
    for b in blocks:
        for _ in range(3):
            b.step()
    torch.cuda.synchronize()
    wants = [[t.clone() for t in b.results()] for b in blocks]
    for b, start in zip(blocks, starts):
        for t, s in zip(b.results(), start):
            t.copy_(s)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(3):
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.step()
    torch.cuda.synchronize()
    for b, want in zip(blocks, wants):
        assert all(torch.equal(t, w) for t, w in zip(b.results(), want))


@pytest.mark.parametrize("xdt", [BF16, F32])
def test_tokens_one_and_a_few_at_a_time(xdt):
    """Decoding: every row of a batch by itself and in groups, each within the bounds of the same formulas."""
    L = qb()
    b = Block(L, 70, xdt)
    b.forward()
    for at, count in [(0, 1), (69, 1), (3, 2), (10, 8), (20, 9), (30, 17), (0, 64)]:
        h, x, a = (t[at:at + count].contiguous() for t in (b.h, b.x, b.a))
        y, g, u = gated.forward(L, h, (b.gate, b.up), "SILU", keep=True)
        gated.check_forward(L, h, (b.gate, b.up), "SILU", y, g, u)
        out = linear.forward(L, a, b.down, b.bias, "NONE", x)
        linear.check_forward(L, a, b.down, b.bias, "NONE", x, out)


# products that take each tile shape, whole and ragged, in one piece and split over their length, with and without
# columns left over whole rounds (the last ones); a last half step in the last piece
PLANS = [(65, 8192, 64), (65, 32, 64), (97, 4128, 129), (256, 1120, 4096), (300, 2080, 1000), (512, 1056, 4099),
         (700, 4000, 700), (1030, 96, 5000), (2048, 160, 2049), (4100, 64, 4352), (2000, 1120, 8500)]


@pytest.mark.parametrize("M,K,N", PLANS)
@pytest.mark.parametrize("xdt", [BF16, F16, F32])
def test_product_plans(M, K, N, xdt):
    """About fifty rows of products of many sizes, of every tile row, against 64 bits."""
    L = qb()
    print(f"[plan] {M} {K} {N} {xdt}", flush=True)
    w = ref.Weight(N, K, oracle.NF4, 64, True, xdt, seed=M)
    x, bias = ref.normal((M, K), M, dtype=xdt), ref.normal((N,), 2)
    y = linear.forward(L, x, w, bias, "SILU")
    rows = sorted({0, 1, 15, 16, 63, 64, M // 2, M // 3, M - 2, M - 1, *range(M - 1, 0, -(M // 40 + 1))})
    at = torch.tensor(rows, device=DEV)
    linear.check_forward(L, x[at], w, bias, "SILU", None, y[at])
    assert y.isfinite().all()
    dy = ref.normal((M, N), 5, 0.1, xdt)
    dx, dz, _ = linear.backward(L, dy, w, dz=True)
    assert torch.equal(dz, dy)
    linear.check_backward(L, dy[at], w, None, "NONE", dx[at], None, None)
    assert dx.isfinite().all()


# few rows through layers whose block constants pass LDS in several parts, blocks that begin inside a row, steps
# filled in part, fewer steps than waves; both numbers of waves, every number of rows a workgroup takes
LONG = [(1, 12320, 20), (4, 24704, 33), (5, 12288, 6200), (8, 36896, 40), (11, 12384, 6161), (16, 24608, 17),
        (17, 49184, 19), (40, 12416, 33), (48, 24576, 16), (64, 12512, 35)]


@pytest.mark.parametrize("M,K,N", LONG)
@pytest.mark.parametrize("nested,blocksize", [(False, 64), (True, 64), (True, 4096)])
@pytest.mark.parametrize("xdt", [BF16, F32])
def test_few_rows_of_long_layers(M, K, N, nested, blocksize, xdt):
    L = qb()
    print(f"[long] {M} {K} {N} {nested} {blocksize} {xdt}", flush=True)
    x = ref.normal((M, K), M, dtype=xdt)
    if N < 6000:
        w = gated.pair(N, K, oracle.NF4, blocksize, nested, xdt, K)
        x = x * (10 / K ** 0.5)
        y, g, u = gated.forward(L, x, w, "SILU", keep=True)
        gated.check_forward(L, x, w, "SILU", y, g, u)
    w = ref.Weight(N, K, oracle.FP4, blocksize, nested, xdt, seed=M)
    linear.check_forward(L, x, w, None, "NONE", None, linear.forward(L, x, w))


@pytest.mark.parametrize("M,K,N", [(66, 8192, 700), (130, 4096, 3001), (200, 6144, 1100), (300, 2080, 2000),
                                   (520, 1056, 3000), (1025, 96, 2500), (2050, 160, 1025), (4100, 64, 2200), (2000, 1120, 4250)])
@pytest.mark.parametrize("xdt", [BF16, F16, F32])
def test_gated_plans(M, K, N, xdt):
    L = qb()
    print(f"[gated plan] {M} {K} {N} {xdt}", flush=True)
    w = gated.pair(N, K, oracle.NF4, 64, True, xdt, seed=M)
    x = ref.normal((M, K), M, 10 / K ** 0.5, dtype=xdt)
    y, g, u = gated.forward(L, x, w, keep=True)
    at = torch.tensor(sorted({0, 1, 16, 64, M - 1, *range(M - 1, 0, -(M // 40 + 1))}), device=DEV)
    gated.check_forward(L, x[at], w, "SILU", y[at], g[at], u[at])
    assert y.isfinite().all()
    dy = ref.normal((M, N), 5, 0.1, xdt)
    dx = gated.backward(L, dy, g, u, w)[0]
    gated.check_backward(L, dy[at], g[at], u[at], w, "SILU", dx[at])
    assert dx.isfinite().all()


@pytest.mark.parametrize("M", [3, 7, 12, 30, 45, 60])
@pytest.mark.parametrize("N", [40, 6150])
@pytest.mark.parametrize("nested", [False, True])
@pytest.mark.parametrize("xdt", [BF16, F16, F32])
def test_rows_kernels(M, N, nested, xdt):
    """Every number of rows a workgroup takes, with 8 and with 16 waves, one weight and two, in every type."""
    L = qb()
    w = gated.pair(N, 160, oracle.FP4, 128, nested, xdt, M)
    x = ref.normal((M, 160), M, 0.8, dtype=xdt)
    y, g, u = gated.forward(L, x, w, "GELU", keep=True)
    gated.check_forward(L, x, w, "GELU", y, g, u)
    bias = ref.normal((N,), 1, dtype=xdt)
    y, z = linear.forward(L, x, w[0], bias, "RELU", keep=True)
    linear.check_forward(L, x, w[0], bias, "RELU", None, y, z)


@pytest.mark.parametrize("M", [1, 16, 17, 32, 33, 48, 49, 64])
@pytest.mark.parametrize("K,N", [(160, 70), (4096, 4200), (1056, 129)])
@pytest.mark.parametrize("nested", [False, True])
@pytest.mark.parametrize("xdt", [BF16, F16])
def test_gradients_of_few_rows(M, K, N, nested, xdt):
    """Both sides of the rows and sizes up to which no transposed weights are written; slices of one tile and many."""
    L = qb()
    w = gated.pair(N, K, oracle.NF4, 64, nested, xdt, M)
    dy, z, u = (ref.normal((M, N), i, 0.5, xdt) for i in range(3))
    linear.check_backward(L, dy, w[0], None, "NONE", linear.backward(L, dy, w[0])[0], None, None)
    dx, _, db = linear.backward(L, dy, w[0], z, "SILU", bias_dt=F32)
    linear.check_backward(L, dy, w[0], z, "SILU", dx, None, db)
    gated.check_backward(L, dy, z, u, w, "GELU", gated.backward(L, dy, z, u, w, "GELU")[0])
