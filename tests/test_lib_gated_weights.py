"""Host-side checks of a gated block's weights: what a plain weight must leave NULL, and what the binding
hands over of a nested one.  No GPU needed, no kernel runs: the pointers are fake aligned addresses."""
import ctypes

import pytest
import torch

A, B, C, D, E = (0x100000 * i for i in range(1, 6))
BF16, NF4 = 2, 1


@pytest.fixture(scope="module")
def qb():
    from bit_optimizer_states_amd import binding
    binding.lib()
    return binding


def forward(qb, gate, up):
    L = qb.lib()
    return L.qb_dequant_gated(A, BF16, 100, 64, ctypes.byref(gate), ctypes.byref(up), NF4, 64, 256, 48, 4, None, None, D,
                              B + 8, 0, None)                  # (the workspace is refused behind the weights' checks)


def backward(qb, gate, up):
    L = qb.lib()
    return L.qb_dequant_gated_backward(A, B, C, BF16, 100, 64, ctypes.byref(gate), ctypes.byref(up), NF4, 64, 256, 48, 4, D,
                                       None, None, B + 8, 0, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_a_weight_is_plain_or_nested(qb, call):
    """Nested constants without their codes are no plain weight, with an absmax or without."""
    plain, nested = qb.qb_weight(B, C, None, None, None), qb.qb_weight(B, None, C, D, E)
    assert call(qb, plain, plain) == call(qb, nested, nested) == qb.QB_EALIGN            # the workspace
    for bad in (qb.qb_weight(B, C, None, D, E), qb.qb_weight(B, C, None, D, None), qb.qb_weight(B, C, None, None, E),
                qb.qb_weight(B, None, None, D, E)):
        for gate, up in ((bad, plain), (plain, bad), (bad, bad)):
            assert call(qb, gate, up) == qb.QB_EINVAL
    for bad in (qb.qb_weight(B, C, C, D, E), qb.qb_weight(B, None, C, None, E), qb.qb_weight(B, None, C, D, None)):
        for gate, up in ((bad, nested), (nested, bad)):
            assert call(qb, gate, up) == qb.QB_EINVAL


def test_the_binding_hands_over_every_part(qb, monkeypatch):
    """absmax beside nested constants reaches the library, which refuses it."""
    place = {}
    monkeypatch.setattr(qb, "_at", lambda t, device: None if t is None else place.setdefault(id(t), 0x100000 + 16 * len(place)))
    codes, absmax = torch.zeros(1536, dtype=torch.uint8), torch.zeros(48)
    dq = qb.qb_dq(C, D, E, 256, None, 0)
    dq.made_of = None
    gate, up, b2 = qb._gated_weights((codes, absmax, dq), (codes, None, dq), NF4, 64, 48, 64, -1)
    assert b2 == 256 and gate.absmax == place[id(absmax)] and gate.codes == up.codes == place[id(codes)]
    assert (gate.c2, gate.absmax2, gate.offset) == (C, D, E) and up.absmax is None
    assert forward(qb, gate, up) == qb.QB_EINVAL and forward(qb, up, gate) == qb.QB_EINVAL
