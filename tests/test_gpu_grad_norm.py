"""GPU: the global gradient norm and clipping by it against exact sums (math.fsum over
binary64 squares, numpy).

Tolerances: a binary64 sum of n squares of binary32 values (the squares are exact) is off by
at most n 2^-53 relative, which is far below the one rounding to binary32 (2^-24) for the
sizes here; the square root halves it.  The scale is taken from the binary32 norm: the
product g * scale is compared with the one that numpy computes from the returned norm, bit
for bit (binary64 quotient, one rounding to binary32, one binary32 product, one rounding)."""
import math

import numpy as np
import pytest
import torch

import linear_reference as ref
from gpu_helpers import DEV, qb

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def norm_of(L, table, count):
    size = L.qb_multi_tensor_grad_norm_workspace_bytes(count)
    ws = torch.full((size + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    norm = torch.full((8,), 7.0, device=DEV)
    L.qb_multi_tensor_grad_norm(table, count, norm[:1], ws[:size] if size else None)
    torch.cuda.synchronize()
    assert (ws[size:] == 0x5A).all() and (norm[1:] == 7.0).all()
    return norm[:1].clone()


def exact_norm(grads):
    return math.sqrt(math.fsum(float((t.detach().cpu().double() ** 2).sum()) for t in grads))


def expected(g, max_norm, norm):
    s = np.float64(max_norm) / (np.float64(norm.item()) + 1e-6)
    s = np.float32(1.0) if s >= 1.0 else np.float32(s)
    return (g.float() * torch.tensor(s, device=DEV)).to(g.dtype)


def check(L, grads, max_norm, in_place=False, offset=0):
    """Gradients are views of guarded buffers, `offset` elements past an aligned address."""
    outs, guards, sources = [], [], []
    for g in grads:
        for to in (sources, outs):
            buf = torch.full((g.numel() + 16,), 7.0, dtype=g.dtype, device=DEV)
            guards.append((buf, offset, g.numel()))
            to.append(buf[offset:offset + g.numel()])
        sources[-1].copy_(g.view(-1))
    count = len(grads)
    table = L.grad_table(list(sources) if in_place else list(zip(sources, outs)))
    norm = norm_of(L, table, count)
    want = exact_norm(grads)
    assert abs(norm.item() - want) <= want * 2.0 ** -24 * 1.001 + 1e-45
    before = [s.clone() for s in sources]
    L.qb_multi_tensor_clip_grads(table, count, max_norm, norm)
    torch.cuda.synchronize()
    for g, s, o, b in zip(grads, sources, outs, before):
        got = s if in_place else o
        assert torch.equal(got, expected(g.view(-1), max_norm, norm))
        if not in_place:
            assert torch.equal(s, b)
    for buf, at, n in guards:
        assert (buf[:at] == 7.0).all() and (buf[at + n:] == 7.0).all()
    return norm


def grads_of(lengths, types, seed, std=1e-3):
    return [ref.normal((n,), seed + i, std, types[i % len(types)]) for i, n in enumerate(lengths)]


@pytest.mark.parametrize("types", [[F32], [F16], [BF16], [BF16, F32, F16]])
@pytest.mark.parametrize("lengths", [[1], [0, 5, 0], [7, 8, 9, 63, 64, 65], [2047, 2048, 2049, 4095, 4096, 4097],
                                     [100003, 1, 50000], [3000000], [129] * 300, [4099] * 121])
@pytest.mark.parametrize("in_place", [False, True])
def test_lengths_and_types(types, lengths, in_place):
    L = qb()
    grads = grads_of(lengths, types, 1, 0.1)
    total = exact_norm(grads)
    for factor, offset in ((0.3, 0), (0.3, 1), (2.0, 0), (1.0, 3)):
        check(L, grads, total * factor, in_place, offset)


def test_within_the_limit_in_place_nothing_changes():
    L = qb()
    grads = grads_of([5000, 33], [F32, BF16], 2)
    kept = [g.clone() for g in grads]
    table = L.grad_table(grads)
    norm = norm_of(L, table, 2)
    L.qb_multi_tensor_clip_grads(table, 2, 1e9, norm)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))


def test_extreme_magnitudes():
    """Squares beyond binary32 in both directions, and a norm beyond it."""
    L = qb()
    for std in (1e-30, 1e30, 1e-42):
        g = ref.normal((5000,), 3, 1.0) * 1e-3 if std == 1e-42 else ref.normal((5000,), 3, std)
        if std == 1e-42:
            g = g * 1e-39                                # subnormal values
        norm = norm_of(L, L.grad_table([g]), 1)
        want = exact_norm([g])
        assert abs(norm.item() - want) <= want * 2.0 ** -24 * 1.001 + 1e-45
    big = torch.full((100000,), 3e38, device=DEV)
    out = torch.empty_like(big)
    table = L.grad_table([(big, out)])
    norm = norm_of(L, table, 1)
    assert norm.item() == math.inf
    L.qb_multi_tensor_clip_grads(table, 1, 1.0, norm)
    torch.cuda.synchronize()
    assert (out == 0.0).all()


@pytest.mark.parametrize("n", [100, 100000])
def test_nan_and_infinity(n):
    L = qb()
    for bad, at in ((math.nan, 0), (math.inf, n - 1), (-math.inf, n // 2)):
        g = ref.normal((n,), 4)
        g[at] = bad
        out = torch.empty_like(g)
        table = L.grad_table([(g, out)])
        norm = norm_of(L, table, 1)
        assert math.isnan(norm.item()) if math.isnan(bad) else norm.item() == math.inf
        L.qb_multi_tensor_clip_grads(table, 1, 1.0, norm)
        torch.cuda.synchronize()
        if math.isnan(bad):
            assert out.isnan().all()
        else:                                            # times zero: NaN at the infinity alone
            assert out[at].isnan() and (out != 0).sum() == 1


def test_nothing():
    L = qb()
    assert norm_of(L, L.grad_table([]), 0).item() == 0.0
    empty = torch.empty(0, device=DEV)
    assert norm_of(L, L.grad_table([empty, empty]), 2).item() == 0.0
    L.qb_multi_tensor_clip_grads(L.grad_table([empty]), 1, 1.0, torch.ones(1, device=DEV))


def test_a_norm_of_several_ranks():
    """Two halves' norms joined by the caller clip as one call over all gradients."""
    L = qb()
    grads = grads_of([5000, 777, 100000, 3], [F32, BF16], 5)
    whole = norm_of(L, L.grad_table(grads), 4)
    parts = [norm_of(L, L.grad_table(grads[i:i + 2]), 2) for i in (0, 2)]
    joined = torch.sqrt(sum(p.double() ** 2 for p in parts)).float()
    assert abs(joined.item() - whole.item()) <= whole.item() * 3 * 2.0 ** -24
    outs = [torch.empty_like(g) for g in grads]
    L.qb_multi_tensor_clip_grads(L.grad_table(list(zip(grads, outs))), 4, 0.01, joined)
    torch.cuda.synchronize()
    assert all(torch.equal(o, expected(g, 0.01, joined)) for g, o in zip(grads, outs))


def test_captured_call_replays():
    L = qb()
    lengths = [300000, 5, 70001] + [100] * 130
    grads = grads_of(lengths, [F32, BF16], 6)
    outs = [torch.empty_like(g) for g in grads]
    table = L.grad_table(list(zip(grads, outs)))
    count = len(grads)
    ws = torch.empty(L.qb_multi_tensor_grad_norm_workspace_bytes(count), dtype=torch.uint8, device=DEV)
    norm = torch.empty(1, device=DEV)

    def step():
        L.qb_multi_tensor_grad_norm(table, count, norm, ws)
        L.qb_multi_tensor_clip_grads(table, count, 0.05, norm)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    del table                                            # the host table is read during the call only
    again = L.grad_table(list(zip(grads, outs)))
    for i in range(4):
        for j, g in enumerate(grads):
            g.mul_(1.5 if (i + j) % 2 else 0.7)
        L.qb_multi_tensor_grad_norm(again, count, norm, ws)
        L.qb_multi_tensor_clip_grads(again, count, 0.05, norm)
        torch.cuda.synchronize()
        want = [norm.clone()] + [o.clone() for o in outs]
        norm.fill_(9.0)
        ws.fill_(0xEE)
        for o in outs:
            o.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([norm] + outs, want))


def test_same_bits_every_run():
    L = qb()
    grads = grads_of([1 << 22, 1000003], [BF16], 7)
    table = L.grad_table(grads)
    first = norm_of(L, table, 2)
    assert all(torch.equal(norm_of(L, table, 2), first) for _ in range(3))


def test_refusals():
    L = qb()
    g = torch.ones(100, device=DEV)
    table = L.grad_table([g])
    norm, ws = torch.ones(1, device=DEV), torch.empty(1 << 14, dtype=torch.uint8, device=DEV)
    for bad in ([g.cpu()], [g.view(10, 10).t()], [(g, g[:50])], [(g, g.half())], [g.double()]):
        with pytest.raises((ValueError, TypeError)):
            L.grad_table(bad)
    with pytest.raises(ValueError):
        L.qb_multi_tensor_grad_norm(table, 2, norm, ws)
    with pytest.raises(ValueError):
        L.qb_multi_tensor_grad_norm(table, 1, norm.double(), ws)
    for call, status in ((lambda: L.qb_multi_tensor_grad_norm(table, 1, norm, None), L.QB_EINVAL),
                         (lambda: L.qb_multi_tensor_grad_norm(table, 1, norm, ws[:100]), L.QB_EWORKSPACE),
                         (lambda: L.qb_multi_tensor_clip_grads(table, 1, -1.0, norm), L.QB_EINVAL),
                         (lambda: L.qb_multi_tensor_clip_grads(table, 1, math.nan, norm), L.QB_EINVAL)):
        with pytest.raises(L.QbError) as e:
            call()
        assert e.value.status == status


def test_overlapping_gradients_are_measured_and_not_clipped():
    """The norm may count a gradient twice; clipping would scale it twice or once, by chance."""
    L = qb()
    a, b = torch.full((100,), 3.0, device=DEV), torch.full((100,), 4.0, device=DEV)
    out = torch.empty(200, device=DEV)
    for entries in ([a, a], [a, a[50:]], [(a, out[:100]), (b, out[99:199])], [(a, b), b], [(a[:50], a[25:75])], [a, (b, a)]):
        table = L.grad_table(entries)
        norm = norm_of(L, table, len(entries))
        assert abs(norm.item() - exact_norm([e[0] if isinstance(e, tuple) else e for e in entries])) < 1e-4
        with pytest.raises(ValueError, match="overlap"):
            L.qb_multi_tensor_clip_grads(table, len(entries), 1.0, norm)
    for entries in ([a[:50], a[50:]], [(a, out[:100]), (b, out[100:])], [(a, out[:100]), (a, out[100:])], [a, a[:0], b]):
        L.qb_multi_tensor_clip_grads(L.grad_table(entries), len(entries), 1.0, torch.ones(1, device=DEV))
    one = torch.ones(1, device=DEV)             # the scale is 1 / (1 + 1e-6): a was clipped twice in place, b once
    assert torch.equal(a, expected(expected(torch.full_like(a, 3.0), 1.0, one), 1.0, one))
    assert torch.equal(b, expected(torch.full_like(b, 4.0), 1.0, one))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lengths", [[64] * 500, [1, 2, 3, 4097, 5, 0, 8192, 1, 0, 30001], [70000, 1, 70000], [4096, 0, 0, 4096]])
def test_neighbours_of_a_bucket(lengths, in_place):
    """Views that lie next to each other, in order, backwards and with their outputs apart: the norm of the whole,
    every element scaled once, nothing around them written."""
    L = qb()
    total = sum(lengths)
    for dt in (F32, F16, BF16):
        for order in ("forward", "backward", "outputs apart"):
            flat = ref.normal((total + 32,), 1, 0.1, dt)
            out = flat if in_place else torch.full((total + 16 * len(lengths) + 32,), 7.0, dtype=dt, device=DEV)
            before, entries, at, to = flat.clone(), [], 16, 16
            gap = 8 if order == "outputs apart" and not in_place else 0
            places = []
            for n in lengths:
                entries.append((flat[at:at + n], out[to:to + n]))
                places.append((at, to, n))
                at, to = at + n, to + n + gap
            if order == "backward":
                entries.reverse()
            table = L.grad_table(entries)
            norm = norm_of(L, table, len(entries))
            want = exact_norm([before[16:16 + total]])
            assert abs(norm.item() - want) <= want * 2.0 ** -24 * 1.001
            L.qb_multi_tensor_clip_grads(table, len(entries), want / 2, norm)
            torch.cuda.synchronize()
            whole = torch.full_like(out, 7.0) if not in_place else before.clone()
            for at, to, n in places:
                whole[to:to + n] = expected(before[at:at + n], want / 2, norm)
            assert torch.equal(out, whole) and (in_place or torch.equal(flat, before)), (dt, order)


def test_neighbours_of_two_types():
    """A bf16 gradient whose end is where an fp32 one begins."""
    L = qb()
    raw = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    a, b = raw[:2048].view(BF16), raw[2048:].view(F32)
    a.copy_(ref.normal((1024,), 1, dtype=BF16))
    b.copy_(ref.normal((512,), 2))
    old = [a.clone(), b.clone()]
    table = L.grad_table([a, b])
    norm = norm_of(L, table, 2)
    assert abs(norm.item() - exact_norm(old)) <= exact_norm(old) * 2.0 ** -24 * 1.001
    L.qb_multi_tensor_clip_grads(table, 2, 1.0, norm)
    assert torch.equal(a, expected(old[0], 1.0, norm)) and torch.equal(b, expected(old[1], 1.0, norm))
