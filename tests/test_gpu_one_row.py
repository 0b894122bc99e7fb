"""One row has no pitch: [1, d] tensors of any stride between rows, as transposes of columns and slices have them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expand_token_adapter_amd as lb


def _one(t):
    """t [1, d] as the transpose of a column (strides 1, 1), and as a row of a buffer whose width is no multiple of 8."""
    column = t.view(-1, 1).clone().t()
    wide = torch.zeros(2, t.shape[1] + 3, dtype=t.dtype, device=t.device)
    row = wide[:1, : t.shape[1]]
    row.copy_(t)
    assert column.is_contiguous() and column.stride() == (1, 1) and row.stride(0) % 8
    return column, row


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_row_of_any_stride(dtype):
    d, n = 264, 136
    x = torch.randn(1, d, device="cuda").to(dtype)
    w = lb.lora_quant_weight_mx(torch.randn(n, d, device="cuda"))
    q = lb.lora_quant_rows_mx(x)
    y = lb.lora_base_product_mx(q, w, dtype=dtype)
    seg = lb.lora_expert_segments(torch.tensor([[2]], dtype=torch.int32, device="cuda"), 3)
    we = lb.lora_quant_weight_mx(torch.randn(3, n, d, device="cuda"))
    ye = lb.lora_expert_product_mx(q, we, seg, dtype=dtype)
    r = torch.rand(1, 1, device="cuda")
    d_o, dw = lb.lora_expert_combine_backward(x, x.flip(1), r, seg)
    w8 = lb.lora_quant_weight(torch.randn(n, d, device="cuda"))
    table = lb.AdapterTable([torch.randn(16, d, device="cuda").to(dtype)], [torch.randn(n, 16, device="cuda").to(dtype)], [0.5])
    ids = lb.lora_segments_build(torch.zeros(1, dtype=torch.int32, device="cuda"), 1)
    delta = torch.zeros(1, n, dtype=dtype, device="cuda")
    lb.lora_forward(x, table, ids, delta)
    for i in range(2):
        xi = _one(x)[i]
        q8 = lb.lora_quant_rows(xi)
        assert torch.equal(q8.codes, lb.lora_quant_rows(x).codes)
        out = lambda t: _one(torch.zeros_like(t))[i]
        assert torch.equal(lb.lora_dequant_rows(q8, out=out(x)), lb.lora_dequant_rows(q8, dtype))
        assert torch.equal(lb.lora_base_product(q8, w8, y=out(y)), lb.lora_base_product(q8, w8, dtype=dtype))
        yi = out(y)
        lb.lora_forward(xi, table, ids, yi)
        assert torch.equal(yi, delta)
        qi = lb.lora_quant_rows_mx(xi)
        assert torch.equal(qi.codes, q.codes) and torch.equal(qi.scales, q.scales)
        assert torch.equal(lb.lora_dequant_rows_mx(q, out=out(x)), lb.lora_dequant_rows_mx(q, dtype))
        assert torch.equal(lb.lora_base_product_mx(q, w, y=out(y)), y)
        assert torch.equal(lb.lora_expert_product_mx(q, we, seg, y=out(ye)), ye)
        assert torch.equal(lb.lora_expert_gather(xi, seg, y=out(x)), x)
        assert torch.equal(lb.lora_expert_gather_backward(xi, seg, dx=out(x)), x)
        assert torch.equal(lb.lora_expert_combine(xi, r, seg, y=out(x)), lb.lora_expert_combine(x, r, seg))
        got = lb.lora_expert_combine_backward(xi, _one(x.flip(1))[i], r, seg, d_o=out(x))
        assert torch.equal(got[0], d_o) and torch.equal(got[1], dw)
