"""The 4-bit and expert calls together, as a mixture-of-experts layer of a fine-tuning step uses them:

    forward   choices sorted; x to its experts; up = W1_e x (+ adapters on the sorted rows); h = relu(up)^2 in the
              caller's hands; out = W2_e h; y += sum_j w_j out_j
    backward  d_out, dw; dh = W2_e^T d_out; dup; adapters' dA, dB, dX; dx_rows += W1_e^T dup; dx = sum of a token's rows

against the layer in 64 bits on the same codes, in a captured graph, on two streams, and repeated."""
import numpy as np
import pytest
import torch

import mx_helpers as mh
import quant_helpers as qh

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expand_token_adapter_amd as lb


def _f64(t):
    return t.detach().double().cpu().numpy()


class Layer:
    """Weights, buffers and plans that a program keeps; step() runs one forward and backward into them."""

    def __init__(self, T=70, k=2, E=6, d=264, f=328, ranks=(8, 16, 4), bits=8, seed=3):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)
        dev = torch.device("cuda")
        self.T, self.k, self.E, self.d, self.f, self.bits = T, k, E, d, f, bits
        W1, W2 = (0.06 * rnd(E, f, d)).to(dev), (0.06 * rnd(E, d, f)).to(dev)
        self.w1, self.w1t = lb.lora_quant_weight_mx(W1), lb.lora_quant_weight_mx(W1, transpose=True)
        self.w2, self.w2t = lb.lora_quant_weight_mx(W2), lb.lora_quant_weight_mx(W2, transpose=True)
        self.A = [(0.1 * rnd(r, d)).to(dev) for r in ranks]
        self.B = [(0.1 * rnd(f, r)).to(dev) for r in ranks]
        self.table = lb.AdapterTable(self.A, self.B, [1.0, 0.5, -2.0])
        self.dA, self.dB = [torch.zeros_like(a) for a in self.A], [torch.zeros_like(b) for b in self.B]
        self.grads = lb.GradTable(self.dA, self.dB)
        self.x, self.dy = rnd(T, d).to(dev), rnd(T, d).to(dev)
        self.w = torch.rand(T, k, generator=g).to(dev)
        self.ids = torch.from_numpy(mh.random_choices(T, k, E, seed, drop=0.1)).to(dev)
        self.adapter = torch.randint(-1, 3, (T,), generator=g, dtype=torch.int32).to(dev)  # of each token
        R = T * k
        z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device=dev)
        self.seg = lb.ExpertSegments(T, k, E, dev)
        self.row_ids = z(R + 1, dtype=torch.int32)
        self.aseg = lb.Segments(R, 3, dev)
        self.rows, self.up, self.out = z(R, d), z(R, f), z(R, d)
        self.d_out, self.dh, self.drows = z(R, d), z(R, f), z(R, d)
        self.v = z(R, 16)
        self.y, self.dx, self.dw = z(T, d), z(T, d), z(T, k)
        save = (lambda n: lb.QuantRows.empty(R, n, dev)) if bits == 8 else (lambda n: lb.MxRows.empty(R, n, dev))
        self.q = [save(d), save(f), save(d), save(f)]
        torch.cuda.synchronize()

    def step(self):
        save = lb.lora_quant_rows if self.bits == 8 else lb.lora_quant_rows_mx
        seg = lb.lora_expert_segments(self.ids, self.E, out=self.seg)
        lb.lora_expert_gather(self.x, seg, y=self.rows)
        # the adapter of every sorted row is its token's (the last place takes the choices without an expert)
        self.row_ids.fill_(-1)
        at = torch.where(seg.pos < 0, len(self.row_ids) - 1, seg.pos).view(-1).long()
        self.row_ids.scatter_(0, at, self.adapter.repeat_interleave(self.k))
        aseg = lb.lora_segments_build(self.row_ids[:-1], 3, out=self.aseg)
        lb.lora_expert_product_mx(save(self.rows, out=self.q[0]), self.w1, seg, y=self.up)
        lb.lora_shrink(self.rows, self.table, aseg, v=self.v)
        lb.lora_expand_add(self.v, self.table, aseg, self.up)
        h = torch.relu(self.up).square()
        lb.lora_expert_product_mx(save(h, out=self.q[1]), self.w2, seg, y=self.out)
        self.y.copy_(self.x)  # a residual
        lb.lora_expert_combine(self.out, self.w, seg, y=self.y, accumulate=True)
        # backward
        lb.lora_expert_combine_backward(self.dy, self.out, self.w, seg, d_o=self.d_out, dw=self.dw)
        lb.lora_expert_product_mx(save(self.d_out, out=self.q[2]), self.w2t, seg, y=self.dh)
        dup = self.dh * 2 * torch.relu(self.up)
        lb.lora_expert_product_mx(save(dup, out=self.q[3]), self.w1t, seg, y=self.drows)
        for t in self.dA + self.dB:
            t.zero_()
        lb.lora_backward(self.rows, dup, self.table, self.grads, aseg, dx=self.drows, v_saved=self.v)
        self.dx.copy_(self.dy)  # the residual's
        lb.lora_expert_gather_backward(self.drows, seg, dx=self.dx, accumulate=True)

    def outputs(self):
        return [self.y, self.dx, self.dw, self.up, self.out, self.dh, self.drows] + self.dA + self.dB


def _weights(w):
    return mh.values(mh.unpack(w.codes.cpu().numpy()), w.scales.cpu().numpy(), w.d_in).reshape(w.experts, w.d_out, w.d_in)


def _rows(q):
    if isinstance(q, lb.QuantRows):
        return qh.values(q.codes.cpu().numpy(), q.scales.cpu().numpy()[:, : -(-q.d // 128)], q.d)
    return mh.values(mh.unpack(q.codes.cpu().numpy()), q.scales.cpu().numpy(), q.d)


def _near(got, want, what, tol=2e-5):
    err = np.abs(_f64(got) - want).max() / max(np.abs(want).max(), 1e-30)
    assert err <= tol, (what, err)


@pytest.mark.parametrize("bits", [4, 8])
def test_step_against_64_bits(bits):
    """Every product from the codes that the step saved, everything else from its formula: fp32 sums of at most 328
    products, each off by at most 2^-23 of the magnitudes added so far, relative to the largest value (2e-5)."""
    L = Layer(bits=bits)
    L.step()
    torch.cuda.synchronize()
    assert int(L.seg.err.item()) == 0 and int(L.aseg.err.item()) == 0
    off, perm, pos = mh.sort_choices(L.ids.cpu().numpy(), L.E)
    n = len(perm)
    tok = perm // L.k
    x, dy, w, ad = _f64(L.x), _f64(L.dy), _f64(L.w), L.adapter.cpu().numpy()
    w1, w2, w1t, w2t = map(_weights, (L.w1, L.w2, L.w1t, L.w2t))
    assert np.array_equal(w1t, w1.transpose(0, 2, 1)) and np.array_equal(w2t, w2.transpose(0, 2, 1))
    which = np.repeat(np.arange(L.E), np.diff(off))
    prod = lambda rows, W: np.stack([W[e] @ r for e, r in zip(which, rows)])
    A, B, s = [_f64(a) for a in L.A], [_f64(b) for b in L.B], [1.0, 0.5, -2.0]
    rows = x[tok]
    assert np.array_equal(_f64(L.rows)[:n], rows)
    q = [_rows(v)[:n] for v in L.q]
    up = prod(q[0], w1)
    for i, t in enumerate(tok):
        if ad[t] >= 0:
            up[i] += s[ad[t]] * B[ad[t]] @ (A[ad[t]] @ rows[i])
    _near(L.up[:n], up, "up")
    out = prod(q[1], w2)
    _near(L.out[:n], out, "out")
    out, up = _f64(L.out)[:n], _f64(L.up)[:n]
    y, dw, d_out = x.copy(), np.zeros((L.T, L.k)), np.zeros((n, L.d))
    for t in range(L.T):
        for j in range(L.k):
            p = pos[t, j]
            if p >= 0:
                y[t] += w[t, j] * out[p]
                dw[t, j] = dy[t] @ out[p]
                d_out[p] = w[t, j] * dy[t]
    _near(L.y, y, "y")
    _near(L.dw, dw, "dw")
    _near(L.d_out[:n], d_out, "d_out")
    _near(L.dh[:n], prod(q[2], w2t), "dh")
    dup = _f64(L.dh)[:n] * 2 * np.maximum(up, 0)
    drows = prod(q[3], w1t)
    dA, dB = [np.zeros_like(a) for a in A], [np.zeros_like(b) for b in B]
    for i, t in enumerate(tok):
        a = ad[t]
        if a >= 0:
            gi = B[a].T @ dup[i]
            drows[i] += s[a] * A[a].T @ gi
            dA[a] += s[a] * np.outer(gi, rows[i])
            dB[a] += s[a] * np.outer(dup[i], A[a] @ rows[i])
    _near(L.drows[:n], drows, "drows")
    for i in range(3):
        _near(L.dA[i], dA[i], f"dA{i}")
        _near(L.dB[i], dB[i], f"dB{i}")
    dx = dy.copy()
    got = _f64(L.drows)
    for t in range(L.T):
        for j in range(L.k):
            if pos[t, j] >= 0:
                dx[t] += got[pos[t, j]]
    _near(L.dx, dx, "dx")


@pytest.mark.parametrize("T,bits", [(3, 8), (70, 4), (400, 8)])
def test_captured_step_replays_on_new_inputs(T, bits):
    L = Layer(T=T, bits=bits)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        L.step()  # (allocates what the wrappers keep)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        L.step()
    other = Layer(T=T, bits=bits, seed=8)  # eager work and other tensors between the replays
    for r in range(4):
        L.x.normal_(generator=torch.Generator(device="cuda").manual_seed(r))
        L.ids.copy_(torch.from_numpy(mh.random_choices(T, L.k, L.E, 100 + r, drop=0.2)))  # other experts, other row counts
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in L.outputs()]
        other.step()
        L.step()
        torch.cuda.synchronize()
        for a, b in zip(got, L.outputs()):
            assert torch.equal(a, b), r


def test_two_streams_at_once_and_repeats():
    layers = [Layer(T=t, bits=b, seed=s) for t, b, s in ((300, 8, 1), (170, 4, 2))]
    want = []
    for L in layers:
        L.step()
        torch.cuda.synchronize()
        want.append([t.clone() for t in L.outputs()])
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        for L, s in zip(layers, streams):
            with torch.cuda.stream(s):
                L.step()
    torch.cuda.synchronize()
    for L, w in zip(layers, want):
        for a, b in zip(L.outputs(), w):
            assert torch.equal(a, b)


def test_a_step_without_a_choice_leaves_the_residual():
    L = Layer()
    L.ids.fill_(-1)
    for t in (L.rows, L.out, L.d_out, L.drows):
        t.fill_(float("nan"))  # what no choice names is not read
    L.step()
    assert torch.equal(L.y, L.x) and torch.equal(L.dx, L.dy) and not L.dw.any()
    assert all(not t.any() for t in L.dA + L.dB)
