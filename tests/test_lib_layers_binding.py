"""Host: qb_dequant_embedding's binding refuses code and scale tensors that the
kernel would read past their ends, before any pointer is looked at.  No GPU needed:
host tensors, which are refused as such only when everything else is right."""
import pytest
import torch

F32, F16, U8 = torch.float32, torch.float16, torch.uint8


@pytest.fixture
def qb(monkeypatch):
    from bit_optimizer_states_amd import binding
    binding.lib()
    monkeypatch.setattr(binding, "_ptr", lambda t: None if t is None else t.data_ptr())
    return binding


def call(qb, codes, absmax, dq, rows=10, dim=64, code=None, blocksize=64):
    ids = torch.zeros(4, dtype=torch.int64)
    qb.qb_dequant_embedding(codes, absmax, dq, qb.QB_DYN8 if code is None else code, blocksize, rows, ids,
                            torch.zeros(4, dim))


def test_types_of_codes_and_absmax(qb):
    codes, absmax = torch.zeros(640, dtype=U8), torch.zeros(10)
    with pytest.raises(ValueError, match="device tensor"):
        call(qb, codes, absmax, None)
    for dt in (F16, torch.bfloat16, torch.float64, torch.int32):
        with pytest.raises(ValueError, match="fp32 absmax"):
            call(qb, codes, absmax.to(dt), None)
    for dt in (torch.int32, torch.int8, F32):
        with pytest.raises(ValueError, match="uint8 codes"):
            call(qb, codes.to(dt), absmax, None)


def test_nested_constants(qb):
    """10 x 64 elements in blocks of 64: 10 blocks, one second-level block of 256; 100 x 4096: 6400 and 25."""
    def dq(c2=10, a2=1, off=1, c2t=U8, a2t=F32, offt=F32):
        return qb.make_dq(torch.zeros(c2, dtype=c2t), torch.zeros(a2, dtype=a2t), torch.zeros(off, dtype=offt), 256)

    codes = torch.zeros(640, dtype=U8)
    with pytest.raises(ValueError, match="device tensor"):
        call(qb, codes, None, dq())
    for bad, what in ((dict(c2=9), "dq codes"), (dict(a2=0), "dq absmax2"), (dict(off=0), "dq offset"),
                      (dict(c2t=torch.int32), "dq codes"), (dict(a2t=F16), "dq absmax2"), (dict(offt=F16), "dq offset")):
        with pytest.raises(ValueError, match=what):
            call(qb, codes, None, dq(**bad))
    codes = torch.zeros(100 * 4096 // 2, dtype=U8)
    with pytest.raises(ValueError, match="device tensor"):
        call(qb, codes, None, dq(c2=6400, a2=25), rows=100, dim=4096, code=qb.QB_NF4)
    for bad in (dict(c2=6400, a2=24), dict(c2=6399, a2=25)):
        with pytest.raises(ValueError, match="dq"):
            call(qb, codes, None, dq(**bad), rows=100, dim=4096, code=qb.QB_NF4)
    # one filled in by hand is taken as it is
    with pytest.raises(ValueError, match="device tensor"):
        call(qb, torch.zeros(640, dtype=U8), None, qb.qb_dq(0x1000, 0x1000, 0x1000, 256, None, 0))
