"""Sizes past 2^31 - 1, which the C calls' int32 would take as other numbers (2^32 + 8 as 8): the binding refuses them
before anything is allocated or enqueued.  The tensors are views of a few numbers with strides of zero."""
import pytest
import torch

import expand_token_adapter_amd as lb

BIG = 2 ** 32 + 8


def _view(rows, cols, dtype=torch.bfloat16):
    """[rows, cols] over one row: the stride between rows is 0."""
    return torch.zeros(cols, dtype=dtype).as_strided((rows, cols), (0, 1))


@pytest.fixture(autouse=True)
def cpu(monkeypatch):
    monkeypatch.setattr(lb, "_on_gpu", lambda *ts: None)

    def never(*a, **k):
        raise AssertionError("enqueued")

    monkeypatch.setattr(lb, "_launch", never)
    monkeypatch.setattr(lb, "_launch_on", never)


def test_rows():
    x = _view(BIG, 8)
    for call in (lb.lora_quant_rows, lb.lora_quant_rows_mx, lb.lora_quant_weight, lb.lora_quant_weight_mx):
        with pytest.raises(ValueError, match="2\\^31"):
            call(x)
    with pytest.raises(ValueError, match="2\\^31"):
        lb.lora_quant_weight_mx(x[None])
    codes, scales = _view(BIG, 128, torch.uint8), _view(BIG, 8, torch.uint8)
    for form in (lambda: lb.MxRows(codes, scales, 8), lambda: lb.QuantRows(codes, scales, 8), lambda: lb.MxWeight(codes, scales, BIG, 8),
                 lambda: lb.MxWeight(codes, scales, BIG // 8, 8, experts=8)):
        with pytest.raises(ValueError, match="2\\^31"):
            form()


def test_columns_and_outputs():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    with pytest.raises(ValueError, match="2\\^31"):
        lb.MxRows(u8(2, 256), u8(2, 8), BIG)
    with pytest.raises(ValueError, match="2\\^31"):
        lb.QuantRows(u8(2, 256), u8(2, 8), BIG)
    q = lb.MxRows(u8(4, 128), u8(4, 8), 200)
    with pytest.raises(ValueError, match="2\\^31"):
        lb._matrix("call", _view(BIG, 8), "y", BIG, -1)
    wide = torch.zeros(8).as_strided((4, BIG), (0, 0))  # (strides of contiguous rows are checked first)
    with pytest.raises(ValueError):
        lb.lora_dequant_rows_mx(q, out=wide)


def test_choices_and_rows_of_adapters():
    for T, k, E in ((2 ** 31, 1, 4), (2 ** 30, 2, 4), (1, BIG, 4), (4, 2, BIG)):
        with pytest.raises(ValueError, match="2\\^31"):
            lb.ExpertSegments(T, k, E, torch.device("cpu"))
    with pytest.raises(ValueError, match="2\\^31"):
        lb.Segments(BIG, 4, torch.device("cpu"))
    with pytest.raises(ValueError, match="2\\^31"):
        lb.Segments(4, BIG, torch.device("cpu"))
