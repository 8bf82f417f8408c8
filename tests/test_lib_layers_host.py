"""Host-side checks of the row-wise layers (embedding lookup, layer norm, stable
embedding): arguments are refused before anything is enqueued, sizes of the
workspaces, shape checks of the binding.  No GPU needed, no kernel runs: the
pointers passed as device buffers are fake aligned addresses."""
import ctypes

import pytest
import torch

A, B, C = 0x100000, 0x200000, 0x300000
F32, F16, BF16 = 0, 1, 2
I32, I64 = 0, 1
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def qb():
    from bit_optimizer_states_amd import binding
    binding.lib()
    return binding


def call(f, defaults, **kw):
    args = dict(defaults)
    for k in kw:
        assert k in args, k
    args.update(kw)
    return f(*args.values())


def check(qb, f, defaults, n_name, bad, misaligned):
    """bad: (status, changed arguments); every pointer of `misaligned` off by 8 is QB_EALIGN."""
    assert call(f, defaults, **{n_name: 0}, **({"accumulate": 1} if "accumulate" in defaults else {})) == qb.QB_OK
    for status, kw in bad:
        assert call(f, defaults, **kw) == status, kw
    for name in misaligned:
        assert call(f, defaults, **{name: defaults[name] + 8}) == qb.QB_EALIGN, name


LOOKUP_BAD = [dict(n=-1), dict(n=1 << 31), dict(rows=-1), dict(rows=1 << 31), dict(dim=0), dict(dim=1 << 24),
              dict(idt=2), dict(scale=NAN), dict(scale=INF), dict(scale=1e39)]


def test_embedding_arguments_rejected_before_launch(qb):
    d = dict(table=A, tdt=BF16, rows=100, dim=64, ids=B, idt=I64, n=10, scale=1.0, y=C, ydt=BF16, stream=None)
    bad = [(qb.QB_EINVAL, kw) for kw in LOOKUP_BAD + [dict(tdt=3), dict(ydt=-1), dict(table=None), dict(ids=None),
                                                      dict(y=None)]]
    check(qb, qb.lib().qb_embedding, d, "n", bad, ["table", "ids", "y"])


def test_dequant_embedding_arguments_rejected_before_launch(qb):
    dq = qb.qb_dq(A, A, A, 256, None, 0)
    ref = ctypes.byref
    d = dict(codes=A, absmax=B, dq=None, code=1, blocksize=64, rows=100, dim=64, ids=B, idt=I32, n=10, scale=1.0, y=C,
             ydt=BF16, stream=None)
    bad = [(qb.QB_EINVAL, kw) for kw in LOOKUP_BAD + [
        dict(ydt=3), dict(code=3), dict(code=-1), dict(blocksize=32), dict(blocksize=100), dict(blocksize=8192),
        dict(codes=None), dict(absmax=None), dict(dq=ref(dq)), dict(ids=None), dict(y=None),
        dict(absmax=None, dq=ref(qb.qb_dq(A, A, A, 100, None, 0))),
        dict(absmax=None, dq=ref(qb.qb_dq(None, A, A, 256, None, 0))),
        dict(absmax=None, dq=ref(qb.qb_dq(A, None, A, 256, None, 0))),
        dict(absmax=None, dq=ref(qb.qb_dq(A, A, None, 256, None, 0))),
        dict(rows=(1 << 31) - 1, dim=128)]]                                  # too many blocks
    bad += [(qb.QB_EALIGN, dict(absmax=None, dq=ref(qb.qb_dq(A + 4, A, A, 256, None, 0)))),
            (qb.QB_EALIGN, dict(absmax=None, dq=ref(qb.qb_dq(A, A + 4, A, 256, None, 0)))),
            (qb.QB_EALIGN, dict(absmax=None, dq=ref(qb.qb_dq(A, A, A + 4, 256, None, 0))))]
    check(qb, qb.lib().qb_dequant_embedding, d, "n", bad, ["codes", "absmax", "ids", "y"])


def test_embedding_backward_arguments_rejected_before_launch(qb):
    L = qb.lib()
    ws = L.qb_embedding_workspace_bytes(10, 100, 64)
    d = dict(dy=A, gdt=BF16, ids=B, idt=I64, n=10, rows=100, dim=64, scale=1.0, padding_id=-1, accumulate=0, dtable=C,
             ddt=F32, ws=A, ws_bytes=ws, stream=None)
    bad = [(qb.QB_EINVAL, kw) for kw in LOOKUP_BAD + [
        dict(n=(1 << 30) + 1), dict(rows=(1 << 26) + 1), dict(gdt=3), dict(ddt=3), dict(padding_id=-2), dict(padding_id=1 << 31),
        dict(accumulate=2), dict(accumulate=-1), dict(dy=None), dict(ids=None), dict(dtable=None), dict(ws=None)]]
    bad += [(qb.QB_EWORKSPACE, dict(ws_bytes=ws - 1)), (qb.QB_EWORKSPACE, dict(ws_bytes=0)), (qb.QB_OK, dict(rows=0))]
    check(qb, L.qb_embedding_backward, d, "n", bad, ["dy", "ids", "dtable", "ws"])


def test_layer_norm_arguments_rejected_before_launch(qb):
    d = dict(x=A, xdt=BF16, n=10, dim=64, gamma=B, beta=B, wdt=F32, eps=1e-5, y=C, mean=A, rstd=B, stream=None)
    bad = [(qb.QB_EINVAL, kw) for kw in [
        dict(n=-1), dict(n=1 << 31), dict(dim=0), dict(dim=1 << 24), dict(xdt=3), dict(wdt=3), dict(eps=0.0),
        dict(eps=-1e-5), dict(eps=1e-60), dict(eps=1e-39), dict(eps=NAN), dict(eps=INF), dict(eps=1e39), dict(x=None), dict(y=None)]]
    bad += [(qb.QB_EUNSUPPORTED, dict(wdt=F16)), (qb.QB_EUNSUPPORTED, dict(xdt=F32, wdt=BF16))]
    check(qb, qb.lib().qb_layer_norm, d, "n", bad, ["x", "gamma", "beta", "y", "mean", "rstd"])


def test_layer_norm_backward_arguments_rejected_before_launch(qb):
    L = qb.lib()
    ws = L.qb_layer_norm_workspace_bytes(10, 64)
    d = dict(dy=A, x=B, xdt=BF16, n=10, dim=64, gamma=B, wdt=F32, mean=A, rstd=B, dx=C, dgamma=C, dbeta=C,
             accumulate=0, ws=A, ws_bytes=ws, stream=None)
    bad = [(qb.QB_EINVAL, kw) for kw in [
        dict(n=-1), dict(n=1 << 31), dict(dim=0), dict(dim=1 << 24), dict(xdt=3), dict(wdt=3), dict(accumulate=2),
        dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(ws=None)]]
    bad += [(qb.QB_EUNSUPPORTED, dict(wdt=F16)), (qb.QB_EWORKSPACE, dict(ws_bytes=ws - 1)),
            (qb.QB_EWORKSPACE, dict(ws_bytes=ws - 1, dgamma=None)),
            (qb.QB_OK, dict(dx=None, dgamma=None, dbeta=None))]                      # nothing wanted
    check(qb, L.qb_layer_norm_backward, d, "n", bad,
          ["dy", "x", "gamma", "mean", "rstd", "dx", "dgamma", "dbeta", "ws"])


def test_stable_embedding_arguments_rejected_before_launch(qb):
    d = dict(table=A, tdt=F32, rows=100, dim=64, ids=B, idt=I64, n=10, scale=1.0, gamma=A, beta=A, wdt=F32, eps=1e-5,
             y=C, ydt=BF16, stream=None)
    bad = [(qb.QB_EINVAL, kw) for kw in LOOKUP_BAD + [
        dict(tdt=3), dict(ydt=3), dict(wdt=3), dict(eps=0.0), dict(eps=NAN), dict(table=None), dict(ids=None),
        dict(y=None)]]
    bad += [(qb.QB_EUNSUPPORTED, dict(dim=16385)), (qb.QB_EUNSUPPORTED, dict(wdt=BF16)),
            (qb.QB_EUNSUPPORTED, dict(tdt=BF16, wdt=F16))]
    check(qb, qb.lib().qb_stable_embedding, d, "n", bad, ["table", "ids", "gamma", "beta", "y"])


def test_stable_embedding_backward_arguments_rejected_before_launch(qb):
    L = qb.lib()
    ws = L.qb_stable_embedding_workspace_bytes(10, 100, 64)
    d = dict(dy=A, gdt=BF16, table=B, tdt=F32, rows=100, dim=64, ids=B, idt=I64, n=10, scale=1.0, gamma=A, wdt=F32,
             eps=1e-5, padding_id=-1, accumulate=0, dtable=C, ddt=BF16, dgamma=C, dbeta=C, ws=A, ws_bytes=ws,
             stream=None)
    bad = [(qb.QB_EINVAL, kw) for kw in LOOKUP_BAD + [
        dict(n=(1 << 30) + 1), dict(rows=(1 << 26) + 1), dict(gdt=3), dict(tdt=3), dict(ddt=3), dict(wdt=3), dict(padding_id=-2),
        dict(eps=0.0), dict(accumulate=2), dict(dy=None), dict(table=None), dict(ids=None), dict(dtable=None),
        dict(ws=None)]]
    bad += [(qb.QB_EUNSUPPORTED, dict(dim=16385)), (qb.QB_EUNSUPPORTED, dict(tdt=F16, wdt=BF16)),
            (qb.QB_EWORKSPACE, dict(ws_bytes=ws - 1))]
    check(qb, L.qb_stable_embedding_backward, d, "n", bad,
          ["dy", "table", "ids", "gamma", "dtable", "dgamma", "dbeta", "ws"])


def test_workspace_sizes(qb):
    L = qb.lib()
    # invalid sizes
    for n, rows, dim in ((-1, 10, 8), ((1 << 30) + 1, 10, 8), (1, -1, 8), (1, (1 << 26) + 1, 8), (1, 10, 0)):
        assert L.qb_embedding_workspace_bytes(n, rows, dim) == 0
        assert L.qb_stable_embedding_workspace_bytes(n, rows, dim) == 0
    assert L.qb_stable_embedding_workspace_bytes(1, 10, 16385) == 0
    assert L.qb_layer_norm_workspace_bytes(-1, 8) == 0 and L.qb_layer_norm_workspace_bytes(8, 0) == 0
    # entries of the table, order and ids of the tokens, used and long ids (per class and as lists), two rows of sums per
    # chunk of 32 tokens
    want = sum(-(-4 * words // 256) * 256 for words in (256 * 125 + 1, 16384, 16384, 514, 4 * 16384, 513)) + 2 * 512 * 4096 * 4
    assert L.qb_embedding_workspace_bytes(16384, 32000, 4096) == want
    # partial sums of dgamma and dbeta of at most 256 workgroups, rows padded to 8 elements
    assert L.qb_layer_norm_workspace_bytes(16384, 4093) == 256 * 2 * 4096 * 4
    assert L.qb_layer_norm_workspace_bytes(3, 1) == 3 * 2 * 8 * 4
    assert L.qb_stable_embedding_workspace_bytes(16384, 32000, 4096) >= want
    # sizes grow with every argument
    for f in (L.qb_embedding_workspace_bytes, L.qb_stable_embedding_workspace_bytes):
        for base in ((1, 1, 1), (1000, 300, 77), (1 << 20, 1 << 18, 4096)):
            for i in range(3):
                more = [v * (2 if i == k else 1) + (1 if i == k else 0) for k, v in enumerate(base)]
                assert f(*more) >= f(*base) > 0


def test_binding_checks_shapes_and_devices(qb):
    """Shape errors are raised before any pointer is looked at (host tensors here)."""
    t = torch.zeros(10, 8)
    ids = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="expected"):
        qb.qb_embedding(t, ids, torch.zeros(5, 8))
    with pytest.raises(ValueError, match="expected"):
        qb.qb_embedding(t, ids, torch.zeros(4, 7))
    with pytest.raises(ValueError, match="device tensor"):
        qb.qb_embedding(t, ids, torch.zeros(4, 8))
    with pytest.raises(ValueError, match="y like x"):
        qb.qb_layer_norm(t, None, None, 1e-5, torch.zeros(10, 7))
    with pytest.raises(ValueError, match="weights of 8"):
        qb.qb_layer_norm(t, torch.zeros(7), None, 1e-5, torch.zeros(10, 8))
    with pytest.raises(ValueError, match="share a dtype"):
        qb.qb_layer_norm(t, torch.zeros(8), torch.zeros(8, dtype=torch.float16), 1e-5, torch.zeros(10, 8))
    with pytest.raises(ValueError, match="statistics"):
        qb.qb_layer_norm(t, None, None, 1e-5, torch.zeros(10, 8), mean=torch.zeros(9))
    with pytest.raises(ValueError, match="codes of the whole table"):
        qb.qb_dequant_embedding(torch.zeros(39, dtype=torch.uint8), torch.zeros(2), None, qb.QB_NF4, 64, 10, ids,
                                torch.zeros(4, 8))
    with pytest.raises(ValueError, match="absmax of every block"):
        qb.qb_dequant_embedding(torch.zeros(80, dtype=torch.uint8), torch.zeros(1), None, qb.QB_DYN8, 64, 10, ids,
                                torch.zeros(4, 8))
    with pytest.raises(ValueError, match="dtable like table"):
        qb.qb_stable_embedding_backward(torch.zeros(4, 8), t, ids, None, 1e-5, torch.zeros(9, 8), None, None, t)
