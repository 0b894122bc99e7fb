"""Calls of the 4-bit and expert operators that their documentation allows beside the ordinary ones: scale bytes at both
ends, wide pitches of every operand, rows grouped by lora_segments_build, weights cut from longer ones, sorts captured."""
import numpy as np
import pytest
import torch

import mx_helpers as mh
import quant_helpers as qh

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expand_token_adapter_amd as lb


def _rows(bits, T, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, k, generator=g, device="cuda")
    return lb.lora_quant_rows_mx(x) if bits == 4 else lb.lora_quant_rows(x)


@pytest.mark.parametrize("T", [3, 40, 300])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scales_far_apart_multiply_to_the_same_values(dtype, bits, T):
    """2^a x times 2^-a w is x times w, bit for bit, up to the last scale bytes that are numbers."""
    k, n = 512, 136
    x, w = _rows(bits, T, k, 1), _rows(4, n, k, 2).as_weight()
    x.scales.fill_(127)
    w.scales.fill_(127)
    want = lb.lora_base_product_mx(x, w, dtype=dtype)
    for sx, sw in ((254, 0), (0, 254), (252, 2), (253, 1), (1, 253)):
        x.scales.fill_(sx)
        w.scales.fill_(sw)
        assert torch.equal(lb.lora_base_product_mx(x, w, dtype=dtype), want), (sx, sw)
    # the largest scales on both sides: infinite where the product is, zero where a row has zeros only
    x.scales.fill_(254)
    w.scales.fill_(254)
    x.codes[0] = 0
    got = lb.lora_base_product_mx(x, w, dtype=dtype)
    assert not got[0].any()


@pytest.mark.parametrize("bits", [4, 8])
def test_pitches_of_every_operand(bits):
    T, k, n, E = 90, 520, 136, 3
    x, w = _rows(bits, T, k, 3), _rows(4, E * n, k, 4).as_weight(E)
    ids = torch.from_numpy(mh.random_choices(T, 1, E, 5, drop=0.2)).cuda()
    seg = lb.lora_expert_segments(ids, E)
    rows = int(seg.offsets[-1])
    want = lb.lora_expert_product_mx(x, w, seg, dtype=torch.float32)

    def wide(t, more):
        out = torch.full((t.shape[0], t.shape[1] + more), 0xEE, dtype=torch.uint8, device="cuda")
        out[:, : t.shape[1]] = t
        return out

    xw = lb.MxRows(wide(x.codes, 256), wide(x.scales, 24), k) if bits == 4 else lb.QuantRows(wide(x.codes, 256), wide(x.scales, 12), k)
    ww = lb.MxWeight(wide(w.codes, 384), wide(w.scales, 8), n, k, experts=E)
    y = torch.full((T, n + 24), 7.0, device="cuda")
    lb.lora_expert_product_mx(xw, ww, seg, y=y[:, 8:n + 8])
    assert torch.equal(y[:rows, 8:n + 8], want[:rows])
    assert (y[:, :8] == 7).all() and (y[:, n + 8:] == 7).all() and (y[rows:] == 7).all()
    lb.lora_expert_product_mx(xw, ww, seg, y=y[:, 8:n + 8], accumulate=True)
    assert torch.equal(y[:rows, 8:n + 8], want[:rows] + want[:rows]) and (y[rows:] == 7).all()
    # one expert's weight cut from them
    one = lb.MxWeight(ww.codes[n:2 * n], ww.scales[n:2 * n], n, k)
    a, b = int(seg.offsets[1]), int(seg.offsets[2])
    assert torch.allclose(lb.lora_base_product_mx(xw[a:b], one, dtype=torch.float32), want[a:b], rtol=1e-5, atol=1e-4)


@pytest.mark.parametrize("bits", [4, 8])
def test_rows_grouped_by_adapter_take_their_adapters_weights(bits):
    """Segments of lora_segments_build in place of the choices': the rows sorted by its permutation."""
    T, k, n, E = 50, 264, 72, 4
    ids = torch.randint(-1, E, (T,), dtype=torch.int32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))
    seg = lb.lora_segments_build(ids, E)
    rows = int(seg.offsets[-1])
    x = torch.randn(T, k, device="cuda")
    xs = torch.zeros_like(x)
    xs[:rows] = x[seg.perm[:rows].long()]
    q = lb.lora_quant_rows_mx(xs) if bits == 4 else lb.lora_quant_rows(xs)
    w = lb.lora_quant_weight_mx(torch.randn(E, n, k, device="cuda"))
    got = lb.lora_expert_product_mx(q, w, seg, dtype=torch.float32)
    wv = lb.lora_dequant_rows_mx(w, torch.float32).view(E, n, k).double()
    xv = (lb.lora_dequant_rows_mx if bits == 4 else lb.lora_dequant_rows)(q, torch.float32).double()
    for i in range(rows):
        e = int(ids[seg.perm[i]])
        # 264 products and as many sums in fp32: 2^-24 of the magnitudes each
        assert ((got[i].double() - wv[e] @ xv[i]).abs() <= 2.0 ** -15 * (wv[e].abs() @ xv[i].abs())).all()
    assert not got[rows:].any()


@pytest.mark.parametrize("T,k,E", [(900, 2, 6), (9000, 8, 16), (700, 2, 1500)])
def test_sorts_replay_on_new_choices(T, k, E):
    """Every build of the sort captured, with the rows' way there and back behind it."""
    d = 72
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    x, w = torch.randn(T, d, device="cuda"), torch.rand(T, k, device="cuda")
    seg = lb.ExpertSegments(T, k, E, ids.device)
    rows, y = torch.zeros(T * k, d, device="cuda"), torch.zeros(T, d, device="cuda")

    def run():
        lb.lora_expert_segments(ids, E, out=seg)
        lb.lora_expert_gather(x, seg, y=rows)
        lb.lora_expert_combine(rows, w, seg, y=y)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for r in range(4):
        c = mh.random_choices(T, k, E, r, drop=0.3)
        ids.copy_(torch.from_numpy(c))
        graph.replay()
        torch.cuda.synchronize()
        off, perm, pos = mh.sort_choices(c, E)
        assert np.array_equal(seg.offsets.cpu().numpy(), off) and np.array_equal(seg.pos.cpu().numpy(), pos)
        got = y.clone()
        assert torch.equal(rows[: len(perm)], x[torch.from_numpy(perm // k).cuda().long()])
        run()
        assert torch.equal(y, got)


def test_every_choice_names_one_expert_and_a_token_names_one_twice():
    T, k, E, d = 300, 3, 5, 40
    ids = torch.full((T, k), 2, dtype=torch.int32, device="cuda")
    seg = lb.lora_expert_segments(ids, E)
    assert torch.equal(seg.pos.view(-1), torch.arange(T * k, dtype=torch.int32, device="cuda"))
    x = torch.randn(T, d, device="cuda")
    rows = lb.lora_expert_gather(x, seg)
    assert torch.equal(rows, x.repeat_interleave(k, 0))
    assert torch.equal(lb.lora_expert_gather_backward(rows, seg), x + x + x)


def test_work_on_another_stream_than_the_tensors():
    T, k, E, d, n = 200, 2, 4, 264, 136
    s = torch.cuda.Stream()
    ids = torch.from_numpy(mh.random_choices(T, k, E, 1)).cuda()
    x, w = torch.randn(T, d, device="cuda"), lb.lora_quant_weight_mx(torch.randn(E, n, d, device="cuda"))

    def run():
        seg = lb.lora_expert_segments(ids, E)
        return lb.lora_expert_product_mx(lb.lora_quant_rows_mx(lb.lora_expert_gather(x, seg)), w, seg, dtype=torch.float32)

    want = run()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,d", [(1023, 2, 72), (1024, 2, 72), (1500, 9, 1032), (1100, 3, 2040), (1100, 3, 2048)])
def test_gradients_of_the_combine_for_many_tokens(T, k, d, dtype):
    """A wave or four waves a token, more choices than are taken at a time, tokens that do not fill a workgroup."""
    g = torch.Generator(device="cuda").manual_seed(T + d)
    seg = lb.lora_expert_segments(torch.from_numpy(mh.random_choices(T, k, 5, 3, drop=0.1)).cuda(), 5)
    n, pos = int(seg.offsets[-1]), seg.pos.long()
    dy = torch.randn(T, d, generator=g, device="cuda").to(dtype)
    o = torch.randn(T * k, d, generator=g, device="cuda").to(dtype)
    o[n:] = float("nan")  # of no choice
    w = torch.randn(T, k, generator=g, device="cuda")
    d_o, dw = lb.lora_expert_combine_backward(dy, o, w, seg, d_o=torch.full_like(o, 7))
    on, at = pos >= 0, pos.clamp(min=0)
    assert (d_o[n:] == 7).all() and not dw[~on].any()
    want = (w.unsqueeze(-1) * dy.float().unsqueeze(1)).to(dtype)
    assert torch.equal(d_o[at[on]], want[on])
    # fp32 sums of a lane's columns, then over its wave and the workgroup: d terms, each rounding 2^-24 of what is added so far
    rows = torch.nan_to_num(o.double())[at]
    exact, mag = (dy.double().unsqueeze(1) * rows).sum(-1), (dy.double().unsqueeze(1) * rows).abs().sum(-1)
    assert ((dw.double() - exact).abs()[on] <= (d / 64 + 16) * 2.0 ** -24 * mag[on]).all()


def test_rows_are_not_sorted_or_joined_in_place():
    """With one choice a token the rows there and back have one shape, but not one order."""
    seg = lb.lora_expert_segments(torch.randint(0, 4, (30, 1), dtype=torch.int32, device="cuda"), 4)
    x, w = torch.randn(30, 64, device="cuda"), torch.rand(30, 1, device="cuda")
    for bad in (lambda: lb.lora_expert_gather(x, seg, y=x), lambda: lb.lora_expert_gather_backward(x, seg, dx=x),
                lambda: lb.lora_expert_combine(x, w, seg, y=x),
                lambda: lb.lora_expert_combine_backward(x, x.clone(), w, seg, d_o=x)):
        with pytest.raises(ValueError):
            bad()
    empty = lb.lora_expert_segments(torch.zeros(0, 1, dtype=torch.int32, device="cuda"), 4)
    assert lb.lora_expert_combine(x[:0], w[:0], empty).shape == (0, 64)
