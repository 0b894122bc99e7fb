"""Which calls may have their products cut: 8-bit rows with bfloat16 y, refused otherwise before anything is enqueued."""
import pytest
import torch

import expand_token_adapter_amd as lb
from expand_token_adapter_amd import _abi

FAKE = 0x10000
CUT = _abi.LORA_MX_CUT
BAD, WS, OK = _abi.LORA_ERR_INVALID_ARG, _abi.LORA_ERR_WORKSPACE, _abi.LORA_OK


@pytest.mark.parametrize("experts", [None, 4])
def test_who_may_cut(experts):
    lib = _abi.load()
    w = _abi.LoraQuant(FAKE, 256, FAKE, 16)
    rows = {4: w, 8: _abi.LoraQuant(FAKE, 384, FAKE, 4)}
    seg = _abi.LoraSegments(FAKE, FAKE, FAKE, FAKE, FAKE)

    def call(dtype, x_bits, T=4, y=FAKE):
        x = rows[8 if x_bits & 8 else 4]
        if experts is None:
            return lib.lora_base_product_mx(dtype, x_bits, x, T, 304, w, 136, y, 136, 0, None, 0, None)
        return lib.lora_expert_product_mx(dtype, x_bits, x, T, 304, w, experts, 136, seg, y, 136, 0, None)

    assert call(0, 8 | CUT, T=0) == OK and call(0, 8 | CUT, y=None) == BAD
    if experts is None:
        assert call(0, 8 | CUT) == WS and call(0, 8) == WS and call(1, 8) == WS and call(0, 4) == WS
    for dtype, x_bits in ((1, 8 | CUT), (0, 4 | CUT), (1, 4 | CUT), (0, CUT), (0, 8 | CUT << 1), (0, 12), (0, -8), (0, 8 | -2 ** 31)):
        assert call(dtype, x_bits, T=0) == BAD, (dtype, x_bits)


def test_the_binding_refuses(monkeypatch):
    monkeypatch.setattr(lb, "_on_gpu", lambda *ts: None)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    x4, x8, w = lb.MxRows(u8(6, 128), u8(6, 8), 200), lb.QuantRows(u8(6, 256), u8(6, 4), 200), lb.MxWeight(u8(8, 128), u8(8, 8), 8, 200)
    seg = lb.Segments.__new__(lb.Segments)
    for x, dtype in ((x4, torch.bfloat16), (x4, torch.float32), (x8, torch.float32)):
        with pytest.raises(ValueError, match="cut"):
            lb.lora_base_product_mx(x, w, dtype=dtype, cut=True)
        with pytest.raises(ValueError, match="cut"):
            lb.lora_expert_product_mx(x, w, seg, dtype=dtype, cut=True)
