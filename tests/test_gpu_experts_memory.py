"""Rows to experts and back inside one wider buffer: columns beside each other are no shared memory, overlapping rows
are refused and leave the buffer as it was."""
import pytest
import torch

import mx_helpers as mh

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expand_token_adapter_amd as lb

T, K, E, D = 50, 3, 5, 136


def _seg():
    return lb.lora_expert_segments(torch.from_numpy(mh.random_choices(T, K, E, 4, drop=0.2)).cuda(), E)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_columns_of_one_buffer(dtype):
    seg = _seg()
    g = torch.Generator(device="cuda").manual_seed(1)
    wide = torch.randn(T * K, 4 * D, generator=g, device="cuda").to(dtype)
    w = torch.rand(T, K, generator=g, device="cuda")
    part = lambda i, rows=T * K: wide[:rows, i * D : (i + 1) * D]
    x, dy = part(0, T).clone(), part(1, T).clone()
    n = int(seg.offsets[-1])
    lb.lora_expert_gather(part(0, T), seg, y=part(2))
    rows = lb.lora_expert_gather(x, seg)
    assert torch.equal(part(2)[:n], rows[:n])
    lb.lora_expert_combine(part(2), w, seg, y=part(3, T))
    assert torch.equal(part(3, T), lb.lora_expert_combine(rows, w, seg))
    want, dw = lb.lora_expert_combine_backward(dy, rows, w, seg)
    got = lb.lora_expert_combine_backward(part(1, T), part(2), w, seg, d_o=part(3))
    assert torch.equal(got[0][:n], want[:n]) and torch.equal(got[1], dw)
    in_place = lb.lora_expert_combine_backward(part(1, T), part(2), w, seg, d_o=part(2))
    assert torch.equal(in_place[0][:n], want[:n]) and torch.equal(in_place[1], dw)
    lb.lora_expert_gather_backward(part(2), seg, dx=part(0, T))
    assert torch.equal(part(0, T), lb.lora_expert_gather_backward(want, seg))
    assert torch.equal(part(1, T), dy)


def test_one_row_in_place_has_no_pitch():
    """The C call with one choice: its row over itself, whatever the pitches say."""
    from expand_token_adapter_amd import _abi

    seg = lb.lora_expert_segments(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 1)
    dy, o, w, dw = torch.randn(1, D, device="cuda"), torch.randn(1, D, device="cuda"), torch.rand(1, 1, device="cuda"), torch.zeros(1, 1, device="cuda")
    want = lb.lora_expert_combine_backward(dy, o, w, seg)
    st = torch.cuda.current_stream().cuda_stream
    assert _abi.load().lora_expert_combine_backward(_abi.LORA_F32, dy.data_ptr(), D, o.data_ptr(), D + 8, 1, D, 1, seg.pos.data_ptr(), w.data_ptr(),
                                                    o.data_ptr(), D, dw.data_ptr(), st) == _abi.LORA_OK
    assert torch.equal(o, want[0]) and torch.equal(dw, want[1])


def test_overlapping_rows_are_refused():
    seg = _seg()
    w = torch.rand(T, K, device="cuda")
    buf = torch.randn(2 * T * K, D, device="cuda")
    before = buf.clone()
    many, less, few = buf[: T * K], buf[1 : T * K + 1], buf[T * K - 1 : T * K - 1 + T]
    flat = buf.view(-1)
    skew = flat[: T * K * (D + 8)].view(T * K, D + 8)[:, :D]  # begins where `many` does, with another pitch
    apart = buf[T * K : T * K + T]
    for bad in (lambda: lb.lora_expert_gather(few, seg, y=many), lambda: lb.lora_expert_gather_backward(many, seg, dx=few),
                lambda: lb.lora_expert_combine(many, w, seg, y=few), lambda: lb.lora_expert_combine_backward(few, many.clone(), w, seg, d_o=many),
                lambda: lb.lora_expert_combine_backward(apart, many, w, seg, d_o=less),
                lambda: lb.lora_expert_combine_backward(apart.clone(), many, w, seg, d_o=skew),
                lambda: lb.lora_expert_combine_backward(apart, many, w, seg, dw=flat[: T * K].view(T, K)),
                lambda: lb.lora_expert_combine_backward(apart, many, w, seg, dw=w)):
        with pytest.raises((ValueError, lb.LoraError)):
            bad()
    assert torch.equal(buf, before)
