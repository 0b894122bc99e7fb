"""One gradient of the experts' combine without the other: the same bits as both together, and nothing else touched."""
import pytest
import torch

import mx_helpers as mh

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expand_token_adapter_amd as lb


# four waves a token, one wave a token; up to eight choices and more; tokens that do not fill a workgroup
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,d", [(1, 1, 8), (33, 2, 1160), (211, 9, 520), (300, 17, 72), (1024, 2, 72), (1500, 9, 1032), (1027, 19, 264),
                                   (1100, 3, 2048)])
def test_one_gradient_alone(T, k, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + d)
    seg = lb.lora_expert_segments(torch.from_numpy(mh.random_choices(T, k, 7, 3, drop=0.1)).cuda(), 7)
    dy = torch.randn(T, d, generator=g, device="cuda").to(dtype)
    o = torch.randn(T * k, d, generator=g, device="cuda").to(dtype)
    w = torch.randn(T, k, generator=g, device="cuda")
    d_o, dw = lb.lora_expert_combine_backward(dy, o, w, seg, d_o=torch.full_like(o, 7))
    # d_o alone, without o, and with an o that would spoil what reads it
    for rows in (None, torch.full_like(o, float("nan"))):
        got, none = lb.lora_expert_combine_backward(dy, rows, w, seg, d_o=torch.full_like(o, 7), need_dw=False)
        assert none is None and torch.equal(got, d_o)
    fresh, _ = lb.lora_expert_combine_backward(dy, None, w, seg, need_dw=False)
    n = int(seg.offsets[-1])
    assert torch.equal(fresh[:n], d_o[:n]) and not fresh[n:].any()
    # dw alone: o is left as it is
    kept = o.clone()
    none, got = lb.lora_expert_combine_backward(dy, o, w, seg, need_d_o=False, dw=torch.full_like(w, 7))
    assert none is None and torch.equal(got, dw) and torch.equal(o, kept)
    # d_o over o itself, where o is not read
    got, _ = lb.lora_expert_combine_backward(dy, kept, w, seg, d_o=kept, need_dw=False)
    assert torch.equal(got[:n], d_o[:n]) and torch.equal(got[n:], o[n:])


def test_one_gradient_replays():
    """Captured without the other, replayed on new choices."""
    T, k, d = 1200, 3, 264
    ids = torch.from_numpy(mh.random_choices(T, k, 5, 1)).cuda()
    seg = lb.lora_expert_segments(ids, 5)
    dy, o, w = torch.randn(T, d, device="cuda"), torch.randn(T * k, d, device="cuda"), torch.rand(T, k, device="cuda")
    d_o, dw = torch.zeros_like(o), torch.zeros_like(w)

    def run():
        lb.lora_expert_segments(ids, 5, out=seg)
        d_o.zero_()
        lb.lora_expert_combine_backward(dy, None, w, seg, d_o=d_o, need_dw=False)
        lb.lora_expert_combine_backward(dy, o, w, seg, dw=dw, need_d_o=False)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for r in range(4):
        ids.copy_(torch.from_numpy(mh.random_choices(T, k, 5, 10 + r, drop=0.3)))
        graph.replay()
        torch.cuda.synchronize()
        got = d_o.clone(), dw.clone()
        both = lb.lora_expert_combine_backward(dy, o, w, lb.lora_expert_segments(ids, 5))
        assert torch.equal(got[0], both[0]) and torch.equal(got[1], both[1]), r


def test_refusals():
    seg = lb.lora_expert_segments(torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 3)
    dy, o, w = torch.zeros(4, 16, device="cuda"), torch.zeros(8, 16, device="cuda"), torch.zeros(4, 2, device="cuda")
    for bad in (dict(need_d_o=False, need_dw=False), dict(need_d_o=False, d_o=o.clone()), dict(need_dw=False, dw=w.clone())):
        with pytest.raises(ValueError):
            lb.lora_expert_combine_backward(dy, o, w, seg, **bad)
    with pytest.raises(ValueError):
        lb.lora_expert_combine_backward(dy, None, w, seg)
    with pytest.raises(ValueError):
        lb.lora_expert_combine_backward(dy, None, w, seg, need_d_o=False)
    with pytest.raises(ValueError):
        lb.lora_expert_combine_backward(dy, o[:, :8], w, seg, need_dw=False)
    empty = lb.lora_expert_segments(torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 3)
    got = lb.lora_expert_combine_backward(dy[:0], None, w[:0], empty, need_dw=False)
    assert got[0].shape == (0, 16) and got[1] is None
