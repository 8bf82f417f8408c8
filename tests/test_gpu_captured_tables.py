"""GPU: the multi-tensor calls and the user code's upload captured into graphs: several graphs with tables of
their own, replayed in turns among eager calls with other tables, equal the same calls made eagerly, bit for bit."""
import gc

import pytest
import torch

from gpu_helpers import DEV, qb

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def normal(n, seed, std=1.0, dtype=F32):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(n, generator=g) * std).to(dtype).to(DEV)


def capture(f):
    f()                                                  # loads the kernels and the constant tables
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f()
    return graph


class Optimizer:
    """Tensors of odd lengths, their states and one step over all of them."""

    def __init__(self, L, count, kind, seed, noalloc=False):
        self.L, self.B, self.noalloc = L, 256, noalloc
        lengths = [1 + (i * 977 + seed * 131) % 5000 for i in range(count)]
        two = kind != L.QB_LARS
        self.p = [normal(n, seed + i, 0.02) for i, n in enumerate(lengths)]
        self.g = [normal(n, seed + 7 * i, 1e-3, BF16) for i, n in enumerate(lengths)]
        codes = lambda n: torch.full((n,), 127, dtype=torch.uint8, device=DEV)  # noqa: E731
        blocks = lambda n: torch.zeros(-(-n // self.B), device=DEV)  # noqa: E731
        self.m, self.am = [codes(n) for n in lengths], [blocks(n) for n in lengths]
        self.v, self.av = ([codes(n) for n in lengths], [blocks(n) for n in lengths]) if two else ([None] * count,) * 2
        if noalloc:
            self.hp, self.ws = L.hparams(lr=1e-2, step=3), None
        else:
            self.hp = L.optim_hparams(kind, 1e-2, weight_decay=0.01, step=3, trust_coefficient=0.01)
            self.ws = torch.empty(L.qb_optimizer_workspace_bytes(self.hp, self.table(), count, self.B), dtype=torch.uint8,
                                  device=DEV)

    def table(self):
        return self.L.tensor_table(list(zip(self.p, self.g, self.m, self.v, self.am, self.av)))

    def step(self):
        table = self.table()                             # (the library reads it during the call only)
        if self.noalloc:
            self.L.qb_multi_tensor_step_noalloc(table, len(self.p), self.L.QB_BF16, self.B, self.hp)
        else:
            self.L.qb_multi_tensor_optimizer_step(self.hp, table, len(self.p), self.L.QB_BF16, self.B, self.ws)

    def state(self):
        return [t for ts in (self.p, self.m, self.v, self.am, self.av) for t in ts if t is not None]


def in_turns(graphs, steps, states, change, others, turns=4):
    """Each turn: the steps made eagerly, then from the same state by their graphs, with `others` (eager calls that
    use the same host buffers for tables of their own) before each replay."""
    for turn in range(turns):
        change(turn)
        starts = [[t.clone() for t in s()] for s in states]
        for f in steps:
            f()
        torch.cuda.synchronize()
        wants = [[t.clone() for t in s()] for s in states]
        for s, start in zip(states, starts):
            for t, c in zip(s(), start):
                t.copy_(c)
        order = list(range(len(graphs)))
        for i in order if turn % 2 else order[::-1]:
            others()
            gc.collect()
            graphs[i].replay()
        torch.cuda.synchronize()
        for s, want in zip(states, wants):
            assert all(torch.equal(t, w) for t, w in zip(s(), want)), turn


@pytest.mark.parametrize("kind", ["QB_ADAMW", "QB_ADAM", "QB_LAMB", "QB_LARS"])
def test_optimizer_steps(kind):
    """Tables of one launch's words and of many."""
    L = qb()
    k = getattr(L, kind)
    parts = [Optimizer(L, c, k, 10 * c) for c in (3, 200, 60)]
    other = [Optimizer(L, c, k, 5 + c) for c in (7, 900)]
    graphs = [capture(p.step) for p in parts]

    def change(turn):
        for p in parts:
            for i, g in enumerate(p.g):
                g.copy_(normal(g.numel(), 1000 * turn + i, 1e-3, BF16))

    in_turns(graphs, [p.step for p in parts], [p.state for p in parts], change, lambda: [o.step() for o in other])


def test_steps_without_a_workspace():
    """Two graphs whose tables share the library's scratch."""
    L = qb()
    parts = [Optimizer(L, c, L.QB_ADAMW, c, noalloc=True) for c in (4, 300)]
    other = Optimizer(L, 700, L.QB_ADAMW, 1, noalloc=True)
    graphs = [capture(p.step) for p in parts]

    def change(turn):
        for p in parts:
            for i, g in enumerate(p.g):
                g.copy_(normal(g.numel(), 1000 * turn + i, 1e-3, BF16))

    in_turns(graphs, [p.step for p in parts], [p.state for p in parts], change, other.step)


class Weights:
    """Tensors that are quantized to NF4 and back in grouped calls."""

    def __init__(self, L, count, nested, seed):
        self.L, self.nested = L, nested
        lengths = [2 + (i * 1931 + seed * 71) % 6000 for i in range(count)]
        self.x = [normal(n, seed + i) for i, n in enumerate(lengths)]
        blocks = [-(-n // 64) for n in lengths]
        byte = lambda n: torch.zeros(n, dtype=torch.uint8, device=DEV)  # noqa: E731
        self.codes = [byte((n + 1) // 2) for n in lengths]
        self.y = [torch.zeros(n, dtype=BF16, device=DEV) for n in lengths]
        if nested:
            self.parts = [(byte(b), torch.zeros(-(-b // 256), device=DEV), torch.zeros(4, device=DEV)) for b in blocks]
            self.absmax = [None] * count
        else:
            self.absmax, self.parts = [torch.zeros(b, device=DEV) for b in blocks], []
        table = self.quant_table()
        self.ws = torch.empty(L.qb_multi_tensor_quantize_workspace_bytes(table, count, 64), dtype=torch.uint8, device=DEV)
        self.ws2 = torch.empty(L.qb_multi_tensor_workspace_bytes(count), dtype=torch.uint8, device=DEV)

    def dqs(self):
        return [self.L.make_dq(*p, 256) for p in self.parts] if self.nested else [None] * len(self.x)

    def quant_table(self):
        return self.L.quant_table([(x, x.numel(), c, a, dq) for x, c, a, dq in zip(self.x, self.codes, self.absmax, self.dqs())])

    def step(self):
        L, count = self.L, len(self.x)
        L.qb_multi_tensor_quantize(self.quant_table(), count, L.QB_F32, L.QB_NF4, 64, 256, self.ws)
        table = L.dequant_table([(c, a, dq, y.numel(), y) for c, a, dq, y in zip(self.codes, self.absmax, self.dqs(), self.y)])
        L.qb_multi_tensor_dequantize(table, count, L.QB_NF4, 64, 256, L.QB_BF16, self.ws2)

    def state(self):
        return self.codes + self.y + [t for t in self.absmax if t is not None] + [t for p in self.parts for t in p[:2]]


@pytest.mark.parametrize("nested", [False, True])
def test_grouped_quantize_and_dequantize(nested):
    L = qb()
    parts = [Weights(L, c, nested, c) for c in (2, 150)]
    other = Weights(L, 400, nested, 3)
    graphs = [capture(p.step) for p in parts]

    def change(turn):
        for p in parts:
            for i, x in enumerate(p.x):
                x.copy_(normal(x.numel(), 1000 * turn + i))

    in_turns(graphs, [p.step for p in parts], [p.state for p in parts], change, other.step)


def test_user_code():
    """A captured upload of a code writes the values that it was given."""
    L = qb()
    codes = [[(i - 128) / 128.0 * s for i in range(256)] for s in (1.0, 0.5, 0.25)]
    tables = [torch.zeros(L.qb_code_table_bytes(), dtype=torch.uint8, device=DEV) for _ in codes]
    graphs = [capture(lambda c=c, t=t: L.qb_prepare_code(c, t)) for c, t in zip(codes[:2], tables)]
    wants = [t.clone() for t in tables[:2]]
    assert not torch.equal(*wants)
    for _ in range(3):
        for g, t, want in zip(graphs, tables, wants):
            t.zero_()
            L.qb_prepare_code(codes[2], tables[2])
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(t, want)


@pytest.mark.parametrize("tokens", [40, 1100])
@pytest.mark.parametrize("xdt", [BF16, F32])
def test_whole_training_steps(tokens, xdt):
    """Forward, backward, clipping and the optimizer's step in one graph, two of them in turn."""
    from test_gpu_layer_step import ROWS, Block

    L = qb()
    blocks = [Block(L, tokens, xdt), Block(L, tokens + 30, xdt, nested=False)]
    other = Optimizer(L, 300, L.QB_ADAMW, 1)
    graphs = [capture(b.step) for b in blocks]

    def change(turn):
        for b in blocks:
            b.ids.copy_(torch.randint(0, ROWS, b.ids.shape, device=DEV))

    def others():
        other.step()
        for b in blocks:
            b.ws.fill_(0xEE)

    in_turns(graphs, [b.step for b in blocks], [b.results for b in blocks], change, others)
