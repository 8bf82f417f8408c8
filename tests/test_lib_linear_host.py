"""Host-side checks of the 4-bit layers with an epilogue, their gradients and the gradient
norm: arguments are refused before anything is enqueued, workspaces never shrink.  No GPU
needed, no kernel runs: the pointers passed as device buffers are fake aligned addresses."""
import ctypes
import random

import pytest
import torch

A, B, C, D, E = (0x100000 * i for i in range(1, 6))
F32, F16, BF16 = 0, 1, 2
NF4, FP4, DYN8 = 1, 2, 0
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


SIZES_BAD = [dict(xdt=3), dict(xdt=-1), dict(M=-1), dict(M=1 << 31), dict(K=0), dict(K=48), dict(K=1 << 21), dict(N=-1),
             dict(N=1 << 21), dict(code=DYN8), dict(code=3), dict(blocksize=32), dict(blocksize=96), dict(blocksize=8192),
             dict(act=-1), dict(act=5)]


def test_linear_arguments_rejected_before_launch(qb):
    L = qb.lib()
    dq = lambda *a: ctypes.byref(qb.qb_dq(*a, None, 0))  # noqa: E731
    ws = L.qb_dequant_linear_workspace_bytes(BF16, 100, 64, 48)
    d = dict(x=A, xdt=BF16, M=100, K=64, codes=B, absmax=C, dq=None, code=NF4, blocksize=64, N=48, bias=D, bdt=F32, act=1,
             residual=E, z=A, y=E, ws=B, ws_bytes=ws, stream=None)
    bad = [(qb.QB_EINVAL, kw) for kw in SIZES_BAD + [
        dict(x=None), dict(y=None), dict(codes=None), dict(absmax=None), dict(bdt=3), dict(ws=None),
        dict(dq=dq(A, A, A, 256)), dict(absmax=None, dq=dq(None, A, A, 256)), dict(absmax=None, dq=dq(A, None, A, 256)),
        dict(absmax=None, dq=dq(A, A, None, 256)), dict(absmax=None, dq=dq(A, A, A, 100)),
        dict(absmax=C, dq=dq(None, A, A, 256))]]
    bad += [(qb.QB_EUNSUPPORTED, dict(bdt=F16)), (qb.QB_EWORKSPACE, dict(ws_bytes=ws - 1)),
            (qb.QB_EALIGN, dict(absmax=None, dq=dq(A + 4, A, A, 256))),
            (qb.QB_EALIGN, dict(absmax=None, dq=dq(A, A + 4, A, 256))),
            (qb.QB_EALIGN, dict(absmax=None, dq=dq(A, A, A + 4, 256)))]
    bad += [(qb.QB_EALIGN, {k: d[k] + 8}) for k in ("x", "codes", "absmax", "bias", "residual", "z", "y", "ws")]
    for status, kw in bad:
        assert call(L.qb_dequant_linear, d, **kw) == status, kw
    for kw in (dict(M=0), dict(N=0), dict(M=0, x=None, codes=None, y=None, ws=None)):
        assert call(L.qb_dequant_linear, d, **kw) == qb.QB_OK, kw


def test_linear_backward_arguments_rejected_before_launch(qb):
    L = qb.lib()
    ws = L.qb_dequant_linear_backward_workspace_bytes(BF16, 100, 64, 48)
    d = dict(dy=A, z=B, xdt=BF16, M=100, K=64, codes=B, absmax=C, dq=None, code=NF4, blocksize=64, N=48, act=2, dx=D,
             dz=E, dbias=C, bdt=F32, accumulate=0, ws=B, ws_bytes=ws, stream=None)
    bad = [(qb.QB_EINVAL, kw) for kw in SIZES_BAD + [
        dict(N=0), dict(dy=None), dict(z=None), dict(codes=None), dict(absmax=None), dict(bdt=-1), dict(ws=None),
        dict(accumulate=2), dict(accumulate=-1), dict(absmax=None, dq=ctypes.byref(qb.qb_dq(None, A, A, 256, None, 0)))]]
    bad += [(qb.QB_EUNSUPPORTED, dict(bdt=F16)), (qb.QB_EWORKSPACE, dict(ws_bytes=ws - 1)),
            (qb.QB_EINVAL, dict(dx=None, ws=None))]
    bad += [(qb.QB_EALIGN, {k: d[k] + 8}) for k in ("dy", "z", "codes", "absmax", "dx", "dz", "dbias", "ws")]
    for status, kw in bad:
        assert call(L.qb_dequant_linear_backward, d, **kw) == status, kw
    for kw in (dict(M=0, dbias=None), dict(M=0, accumulate=1), dict(dx=None, dz=None, dbias=None)):
        assert call(L.qb_dequant_linear_backward, d, **kw) == qb.QB_OK, kw


def test_gated_arguments_rejected_before_launch(qb):
    L = qb.lib()
    ref = ctypes.byref
    plain, nested = qb.qb_weight(B, C, None, None, None), qb.qb_weight(B, None, C, D, E)
    ws = L.qb_dequant_gated_workspace_bytes(BF16, 100, 64, 48)
    d = dict(x=A, xdt=BF16, M=100, K=64, gate=ref(plain), up=ref(plain), code=NF4, blocksize=64, blocksize2=0, N=48, act=4,
             gate_out=B, up_out=C, y=D, ws=B, ws_bytes=ws, stream=None)
    weights_bad = [(qb.QB_EUNSUPPORTED, dict(up=ref(nested))), (qb.QB_EUNSUPPORTED, dict(gate=ref(nested), blocksize2=64)),
                   (qb.QB_EINVAL, dict(gate=ref(nested), up=ref(nested))),            # blocksize2 0
                   (qb.QB_EINVAL, dict(gate=ref(nested), up=ref(nested), blocksize2=100)),
                   (qb.QB_EINVAL, dict(gate=None)), (qb.QB_EINVAL, dict(up=None)),
                   (qb.QB_EINVAL, dict(up=ref(qb.qb_weight(None, C, None, None, None)))),
                   (qb.QB_EINVAL, dict(up=ref(qb.qb_weight(B, None, None, None, None)))),
                   (qb.QB_EINVAL, dict(gate=ref(qb.qb_weight(B, C, C, D, E)), up=ref(nested), blocksize2=64)),
                   (qb.QB_EINVAL, dict(gate=ref(qb.qb_weight(B, None, C, None, E)), up=ref(nested), blocksize2=64)),
                   (qb.QB_EALIGN, dict(up=ref(qb.qb_weight(B + 8, C, None, None, None)))),
                   (qb.QB_EALIGN, dict(up=ref(qb.qb_weight(B, C + 8, None, None, None))))]
    bad = [(qb.QB_EINVAL, kw) for kw in SIZES_BAD + [dict(x=None), dict(y=None), dict(ws=None)]] + weights_bad
    bad += [(qb.QB_EWORKSPACE, dict(ws_bytes=ws - 1))]
    bad += [(qb.QB_EALIGN, {k: d[k] + 8}) for k in ("x", "gate_out", "up_out", "y", "ws")]
    for status, kw in bad:
        assert call(L.qb_dequant_gated, d, **kw) == status, kw
    for kw in (dict(M=0), dict(N=0)):
        assert call(L.qb_dequant_gated, d, **kw) == qb.QB_OK, kw

    ws = L.qb_dequant_gated_backward_workspace_bytes(BF16, 100, 64, 48)
    d = dict(dy=A, gate_out=B, up_out=C, xdt=BF16, M=100, K=64, gate=ref(plain), up=ref(plain), code=NF4, blocksize=64,
             blocksize2=0, N=48, act=4, dx=D, dgate=E, dup=A, ws=B, ws_bytes=ws, stream=None)
    bad = [(qb.QB_EINVAL, kw) for kw in SIZES_BAD + [dict(N=0), dict(dy=None), dict(gate_out=None), dict(up_out=None),
                                                     dict(ws=None)]] + weights_bad
    bad += [(qb.QB_EWORKSPACE, dict(ws_bytes=ws - 1))]
    bad += [(qb.QB_EALIGN, {k: d[k] + 8}) for k in ("dy", "gate_out", "up_out", "dx", "dgate", "dup", "ws")]
    for status, kw in bad:
        assert call(L.qb_dequant_gated_backward, d, **kw) == status, kw
    for kw in (dict(M=0), dict(dx=None, dgate=None, dup=None)):
        assert call(L.qb_dequant_gated_backward, d, **kw) == qb.QB_OK, kw


def test_gradient_norm_arguments_rejected_before_launch(qb):
    L = qb.lib()
    ws = L.qb_multi_tensor_grad_norm_workspace_bytes(1)

    def table(g=A, out=B, n=100, dtype=BF16):
        return (qb.qb_grad * 1)(qb.qb_grad(g, out, n, dtype))

    norm = dict(grads=table(), count=1, norm=C, ws=D, ws_bytes=ws, stream=None)
    clip = dict(grads=table(), count=1, max_norm=1.0, norm=C, stream=None)
    both = [(qb.QB_EINVAL, dict(grads=table(n=-1))), (qb.QB_EINVAL, dict(grads=table(n=1 << 33))),
            (qb.QB_EINVAL, dict(grads=table(dtype=3))), (qb.QB_EINVAL, dict(grads=table(g=None))),
            (qb.QB_EALIGN, dict(grads=table(g=A + 1))), (qb.QB_EALIGN, dict(grads=table(g=A + 2, dtype=F32))),
            (qb.QB_EINVAL, dict(count=-1)), (qb.QB_EINVAL, dict(grads=None)), (qb.QB_EINVAL, dict(norm=None)),
            (qb.QB_EALIGN, dict(norm=C + 8))]
    for status, kw in both + [(qb.QB_EINVAL, dict(ws=None)), (qb.QB_EALIGN, dict(ws=D + 8)),
                              (qb.QB_EWORKSPACE, dict(ws_bytes=ws - 1))]:
        assert call(L.qb_multi_tensor_grad_norm, norm, **kw) == status, kw
    for status, kw in both + [(qb.QB_EINVAL, dict(grads=table(out=None))), (qb.QB_EALIGN, dict(grads=table(out=B + 1))),
                              (qb.QB_EINVAL, dict(max_norm=-1.0)), (qb.QB_EINVAL, dict(max_norm=NAN)),
                              (qb.QB_EINVAL, dict(max_norm=INF))]:
        assert call(L.qb_multi_tensor_clip_grads, clip, **kw) == status, kw
    assert call(L.qb_multi_tensor_clip_grads, clip, grads=table(g=None, out=None, n=0)) == qb.QB_OK
    assert call(L.qb_multi_tensor_clip_grads, clip, count=0, grads=None) == qb.QB_OK
    assert L.qb_multi_tensor_grad_norm_workspace_bytes(0) == 0


def test_workspaces_never_shrink(qb):
    """Around the rows and widths where a call's form changes, and in every direction at random."""
    L = qb.lib()
    fs = [L.qb_dequant_linear_workspace_bytes, L.qb_dequant_linear_backward_workspace_bytes,
          L.qb_dequant_gated_workspace_bytes, L.qb_dequant_gated_backward_workspace_bytes]
    ms = [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 300, 512, 1000, 4096, 5000, 1 << 20, (1 << 31) - 1]
    ks = [32, 64, 96, 128, 992, 1024, 4096, 11008, (1 << 21) - 32]
    ns = [1, 15, 16, 17, 63, 64, 65, 511, 512, 513, 1001, 4096, 11008, 100000, (1 << 21) - 1]
    for f in fs:
        for dt in (F32, F16, BF16):
            for k in ks:
                for n in ns:
                    sizes = [f(dt, m, k, n) for m in ms]
                    assert sizes == sorted(sizes), (k, n)
                for m in ms:
                    sizes = [f(dt, m, k, n) for n in ns]
                    assert sizes == sorted(sizes), (m, k)
            for m in ms:
                for n in ns:
                    sizes = [f(dt, m, k, n) for k in ks]
                    assert sizes == sorted(sizes), (m, n)
        rng = random.Random(3)
        for _ in range(5000):
            m, k, n = int(2 ** rng.uniform(0, 14)), 32 * int(2 ** rng.uniform(0, 9)), int(2 ** rng.uniform(0, 15))
            small = f(BF16, m, k, n)
            assert small <= f(BF16, m + rng.randrange(100), k + 32 * rng.randrange(5), n + rng.randrange(100))
        assert f(BF16, 10, 33, 10) == 0 and f(5, 10, 64, 10) == 0
    sizes = [L.qb_multi_tensor_grad_norm_workspace_bytes(c) for c in range(1, 2000)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def test_binding_refuses_what_a_kernel_would_read_past(qb):
    """Host tensors: refused as such only when everything else is right."""
    u8, bf16 = torch.uint8, torch.bfloat16
    x, y, codes, absmax = torch.zeros(4, 64, dtype=bf16), torch.zeros(4, 48, dtype=bf16), torch.zeros(1536, dtype=u8), torch.zeros(48)
    d = dict(x=x, codes=codes, absmax=absmax, code=NF4, blocksize=64, N=48, y=y)
    with pytest.raises(ValueError, match="device tensor"):
        qb.qb_dequant_linear(**d)
    for bad, what in ((dict(codes=codes[:1535]), "uint8 codes"), (dict(codes=codes.int()), "uint8 codes"),
                      (dict(absmax=absmax[:47]), "fp32 absmax"), (dict(absmax=absmax.half()), "fp32 absmax"),
                      (dict(y=y[:3]), "y of 4 rows"), (dict(y=y.float()), "y of 4 rows"), (dict(residual=x), "residual"),
                      (dict(z=y[:, :47]), "z of"), (dict(bias=torch.zeros(47)), "bias of 48")):
        with pytest.raises(ValueError, match=what):
            qb.qb_dequant_linear(**{**d, **bad})
    with pytest.raises(TypeError):
        qb.qb_dequant_linear(**{**d, "bias": torch.zeros(48, dtype=torch.float64)})
    b = dict(dy=y, codes=codes, absmax=absmax, code=NF4, blocksize=64, K=64, dx=x)
    for bad, what in ((dict(codes=codes[:1535]), "uint8 codes"), (dict(dx=y), "dx of"), (dict(dz=x), "dz of"),
                      (dict(z=x), "z of"), (dict(dbias=torch.zeros(47)), "dbias of 48"), (dict(), "device tensor")):
        with pytest.raises(ValueError, match=what):
            qb.qb_dequant_linear_backward(**{**b, **bad})
    w = (codes, absmax, None)
    for bad, what in ((dict(up=(codes[:1535], absmax, None)), "uint8 codes"), (dict(gate=(codes, absmax[:3], None)), "fp32 absmax"),
                      (dict(gate_out=x), "gate_out of"), (dict(y=x), "y of"), (dict(), "device tensor")):
        with pytest.raises(ValueError, match=what):
            qb.qb_dequant_gated(**{**dict(x=x, gate=w, up=w, code=NF4, blocksize=64, N=48, y=y), **bad})
    for bad, what in ((dict(up_out=x), "up_out of"), (dict(dx=y), "dx of"), (dict(dup=x), "dup of"), (dict(), "device tensor")):
        with pytest.raises(ValueError, match=what):
            qb.qb_dequant_gated_backward(**{**dict(dy=y, gate_out=y, up_out=y, gate=w, up=w, code=NF4, blocksize=64, K=64, dx=x), **bad})
    with pytest.raises(ValueError, match="out like"):
        qb.grad_table([(x, y)])
    table = qb.grad_table([])
    norm, ws = torch.zeros(1), torch.zeros(64, dtype=u8)
    for bad, what in ((dict(norm=torch.zeros(2)), "one fp32"), (dict(norm=norm.double()), "one fp32"),
                      (dict(count=2), "table of count"), (dict(), "device tensor")):
        with pytest.raises(ValueError, match=what):
            qb.qb_multi_tensor_grad_norm(**{**dict(table=table, count=0, norm=norm, ws=ws), **bad})
        with pytest.raises(ValueError, match=what):
            qb.qb_multi_tensor_clip_grads(**{**dict(table=table, count=0, norm=norm, max_norm=1.0), **bad})
    table.device = 1
    with pytest.raises(ValueError, match="gradients' device 1"):
        qb.qb_multi_tensor_grad_norm(table, 0, norm, ws)
