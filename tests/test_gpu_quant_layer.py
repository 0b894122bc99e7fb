"""The 8-bit calls together, as one layer of a fine-tuning step uses them:

    forward   xq = 8-bit rows of x;  y = W x (base product);  v = A x;  y += s B v
    backward  dX = W^T dY (base product of the 8-bit dY);  dX, dA, dB of the adapters from xq

against the layer in 64 bits on the same codes, in a captured graph, on two
streams, and with a workspace and outputs of the caller's own."""
import numpy as np
import pytest
import torch

import oracle
import workloads

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expand_token_adapter_amd as lb
    import quant_helpers as qh
    from gpu_helpers import TOL, GpuCase, rel_err, to_dev

oracle.set_threads(16)


class Layer:
    """Weights, buffers and plans that a program keeps; step() runs one fine-tuning step into them."""

    def __init__(self, dtype="bf16", ranks=(16, 40, 8), d_in=392, d_out=520, T=211, seed=3):
        rng = np.random.default_rng(seed)
        ids = np.concatenate([np.full(T // 2, 1), rng.integers(-1, len(ranks), size=T - T // 2)]).astype(np.int32)
        self.wl = wl = workloads.custom(ids, list(ranks), d_in, d_out, dtype, seed=seed, scales=[2.0, 0.5, -1.0][:len(ranks)],
                                        ft_start=0, ft_count=T, name="quant-layer")
        self.c = c = GpuCase(wl)
        dev = c.dev
        g = torch.Generator().manual_seed(seed)
        W = (0.05 * torch.randn(d_out, d_in, generator=g)).to(c.x.dtype).to(dev)
        self.w, self.wt = lb.lora_quant_weight(W), lb.lora_quant_weight(W, transpose=True)
        self.x, self.dy = c.x.clone(), to_dev(wl.dy, dtype, dev)
        self.xq, self.dyq = lb.QuantRows.empty(T, d_in, dev), lb.QuantRows.empty(T, d_out, dev)
        self.y = torch.zeros(T, d_out, dtype=c.x.dtype, device=dev)
        self.dx = torch.zeros(T, d_in, dtype=c.x.dtype, device=dev)
        self.v = torch.zeros(T, (max(ranks) + 7) // 8 * 8, device=dev)
        self.dA = [torch.zeros(a.shape, device=dev) for a in wl.A]
        self.dB = [torch.zeros(b.shape, device=dev) for b in wl.B]
        self.grads = lb.GradTable(self.dA, self.dB)
        self.seg = lb.lora_segments_build(c.ids, wl.num_adapters)
        torch.cuda.synchronize()

    def step(self):
        lb.lora_quant_rows(self.x, out=self.xq)
        lb.lora_base_product(self.xq, self.w, y=self.y)
        lb.lora_shrink(self.x, self.c.table, self.seg, v=self.v)
        lb.lora_expand_add(self.v, self.c.table, self.seg, self.y)
        lb.lora_quant_rows(self.dy, out=self.dyq)
        lb.lora_base_product(self.dyq, self.wt, y=self.dx)
        for t in self.dA + self.dB:
            t.zero_()
        lb.lora_backward_quant(self.xq, self.dy, self.c.table, self.grads, self.seg, dx=self.dx, v_saved=self.v)

    def outputs(self):
        # (of the scales the bytes of the blocks; those that round a row up to whole words are not written)
        return [self.y, self.dx, self.xq.codes, self.xq.scales[:, : -(-self.xq.d // 128)], self.dyq.codes,
                self.dyq.scales[:, : -(-self.dyq.d // 128)]] + self.dA + self.dB

    def clear(self):
        for t in self.outputs():
            t.zero_()


def _values(q, cols, rows=1):
    return qh.values(q.codes.cpu().numpy(), q.scales.cpu().numpy()[:, : -(-cols // 128)], cols, rows)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ranks", [(16, 5, 12), (16, 40, 8)])
def test_step_against_64_bits(dtype, ranks):
    L = Layer(dtype, ranks)
    L.step()
    torch.cuda.synchronize()
    assert int(L.seg.err.item()) == 0
    wl = L.wl
    ref = oracle.from_workload(wl)
    xv, dyv, wv = _values(L.xq, wl.d_in), _values(L.dyq, wl.d_out), _values(L.w, wl.d_in, 128)
    y, v = oracle.forward(ref["x"], ref["ids"], ref["ranks"], ref["scales"], ref["A"], ref["B"], xv @ wv.T)
    dx, dA, _, _, _ = oracle.backward(xv, ref["dy"], ref["ids"], ref["ranks"], ref["scales"], ref["A"], ref["B"],
                                      dx0=dyv @ wv)
    _, _, dB, _, _ = oracle.backward(ref["x"], ref["dy"], ref["ids"], ref["ranks"], ref["scales"], ref["A"], ref["B"])
    errs = {"y": rel_err(L.y, y), "dx": rel_err(L.dx, dx)}
    errs |= {f"dA{a}": rel_err(t, dA[a]) for a, t in enumerate(L.dA)}
    errs |= {f"dB{a}": rel_err(t, dB[a]) for a, t in enumerate(L.dB)}
    assert all(e <= TOL[dtype] for e in errs.values()), errs


@pytest.mark.parametrize("T", [5, 211])
def test_captured_step_replays_on_new_inputs(T):
    L = Layer(T=T)
    L.step()  # (allocates what the wrappers keep)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.step()
    other = Layer(T=T, seed=8)  # eager work and other tensors between the replays
    for k in range(4):
        g = torch.Generator(device="cuda").manual_seed(k)
        L.x.copy_(torch.randn(L.x.shape, generator=g, device="cuda"))
        L.dy.copy_(torch.randn(L.dy.shape, generator=g, device="cuda"))
        L.clear()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in L.outputs()]
        other.step()
        L.clear()
        L.step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, L.outputs())), k


def test_two_streams_at_once():
    layers = [Layer(seed=s, ranks=r, T=t) for s, r, t in ((1, (16, 40, 8), 500), (2, (16, 5, 12), 300))]
    want = []
    for L in layers:
        L.step()
        torch.cuda.synchronize()
        want.append([t.clone() for t in L.outputs()])
        L.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(3):
        for L, s in zip(layers, streams):
            with torch.cuda.stream(s):
                L.step()
    torch.cuda.synchronize()
    for L, w in zip(layers, want):
        assert all(torch.equal(a, b) for a, b in zip(L.outputs(), w))


def test_same_bits_every_time():
    L = Layer(T=900, d_in=1160, d_out=776)
    L.step()
    first = [t.clone() for t in L.outputs()]
    for _ in range(5):
        L.clear()
        L.step()
        assert all(torch.equal(a, b) for a, b in zip(L.outputs(), first))


def test_workspaces_of_the_caller_and_their_refusal():
    x = lb.lora_quant_rows(torch.randn(64, 14336, device="cuda"))
    w = lb.lora_quant_weight(torch.randn(136, 14336, device="cuda"))
    need = lb.lora_base_product_workspace_bytes(64, 14336, 136)
    assert need > 16  # a long k over few outputs is split
    want = lb.lora_base_product(x, w)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")  # (its contents do not matter)
    assert torch.equal(lb.lora_base_product(x, w, ws=ws[:need]), want)
    assert (ws[need:] == 255).all()
    with pytest.raises(lb.LoraError):
        lb.lora_base_product(x, w, ws=ws[:need // 4])
    with pytest.raises(lb.LoraError):
        lb.lora_base_product(x, w, ws=ws[8:need + 8])


def test_refusals_of_the_binding():
    dev = "cuda"
    x, w = lb.lora_quant_rows(torch.randn(4, 256, device=dev)), lb.lora_quant_weight(torch.randn(16, 256, device=dev))
    y = torch.zeros(4, 16, device=dev)
    bad = [lambda: lb.lora_base_product(x, lb.lora_quant_weight(torch.randn(16, 128, device=dev))),
           lambda: lb.lora_base_product(x, w, accumulate=True), lambda: lb.lora_base_product(x, w, y=y[:3]),
           lambda: lb.lora_base_product(x, w, y=torch.zeros(4, 24, device=dev)),
           lambda: lb.lora_base_product(x, w, y=y.t()), lambda: lb.lora_base_product(x, w, y=y.cpu()),
           lambda: lb.lora_quant_rows(torch.randn(4, 256, device=dev), out=x[:2]),
           lambda: lb.lora_quant_rows(torch.randn(4, 128, device=dev), out=x),
           lambda: lb.lora_dequant_rows(x, out=torch.zeros(4, 128, device=dev)),
           lambda: lb.lora_quant_weight(torch.randn(16, 256, device=dev), transpose=True, out=w),
           lambda: lb.QuantRows(x.codes[:, :128], x.scales, 256), lambda: lb.QuantRows(x.codes, x.scales[:2], 256),
           lambda: lb.QuantRows(x.codes, x.scales[:, :2], 256), lambda: lb.QuantRows(x.codes.t(), x.scales, 4),
           lambda: lb.QuantRows(x.codes.cpu(), x.scales, 256),
           lambda: lb.QuantRows(torch.zeros(4, 320, dtype=torch.uint8, device=dev), x.scales, 256),
           lambda: lb.QuantWeight(w.codes, w.scales, 200, 256)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: lb.lora_base_product(x, w, y=y.half()), lambda: lb.lora_quant_rows(y.half()),
              lambda: lb.lora_dequant_rows(x, torch.float16), lambda: x[0], lambda: x[::2]):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(lb.LoraError):
        lb.lora_quant_rows(torch.randn(4, 260, device=dev))  # columns not a multiple of 8
    # the backward: rows, columns and types that do not belong together
    L = Layer(T=20)
    args = (L.c.table, L.grads, L.seg)
    L.step()
    for q, kw in ((x, {}), (L.xq[:10], {}), (L.xq, dict(dx=L.dx[:10])), (L.xq, dict(dx=L.dx.float())),
                  (L.xq, dict(v_saved=L.v[:10]))):
        with pytest.raises(ValueError):
            lb.lora_backward_quant(q, L.dy, *args, **kw)
    with pytest.raises(ValueError):
        lb.lora_backward_quant(L.xq, L.dy.float(), *args)
