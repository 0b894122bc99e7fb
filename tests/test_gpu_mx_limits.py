"""Products with a 4-bit weight of every kernel that the choice reaches, stored and added, against 64 bits; the
rounding rule at cancelling outliers; offsets past 32 bits; two graphs over one workspace.

Operands are made of codes and scale bytes directly, so that they hold what rounded data rarely does."""
import numpy as np
import pytest
import torch

import mx_helpers as mh
import mx_plans
import quant_helpers as qh

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expand_token_adapter_amd as lb

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _codes4(rows, k, g, low=120, high=134):
    """(packed codes, scale bytes, values in 64 bits on the GPU, scale factors) of random codes, columns past k zero."""
    pad = qh.pad_up(k, 256)
    c = torch.randint(0, 256, (rows, pad // 2), generator=g, device="cuda").to(torch.uint8)
    c[:, k // 2:] = 0
    s = torch.randint(low, high, (rows, pad // 32), generator=g, device="cuda").to(torch.uint8)
    s[:, -(-k // 32):] = 127
    table = torch.from_numpy(mh.E2M1).cuda()
    f = torch.exp2(s.double() - 127).repeat_interleave(32, 1)[:, :k]
    v = table[torch.stack([c & 15, c >> 4], -1).view(rows, -1).long()][:, :k] * f
    return c, s, v, f


def _codes8(rows, k, g):
    pad = qh.pad_up(k, 128)
    c = torch.randint(0, 127, (rows, pad), generator=g, device="cuda") | (torch.randint(0, 2, (rows, pad), generator=g, device="cuda") << 7)
    c[:, k:] = 0
    s = torch.randint(118, 130, (rows, qh.pad_up(pad // 128, 4)), generator=g, device="cuda").to(torch.uint8)
    table = torch.from_numpy(np.nan_to_num(qh.E4M3)).cuda()
    f = torch.exp2(s.double() - 127)[:, : pad // 128].repeat_interleave(128, 1)[:, :k]
    return c.to(torch.uint8), s, table[c][:, :k] * f, f


def _rows(bits, T, k, g):
    if bits == 4:
        c, s, v, f = _codes4(T, k, g)
        return lb.MxRows(c, s, k), v, f
    c, s, v, f = _codes8(T, k, g)
    return lb.QuantRows(c, s, k), v, f


def _bound(x, w, xf, wf, want, dt, bits, y0=None, parts=1):
    """mx_helpers.product_bound, on the GPU."""
    depth = 128 + -(-x.shape[1] // 128) + parts + 8
    mag = x.abs() @ w.abs().t()
    acc = depth * 2.0 ** -23 * mag + 2.0 ** -126
    if bits == 8 and dt == torch.bfloat16:
        top = [torch.where(m == 0, 0.0, torch.maximum(m.abs(), least * f)).view(m.shape[0], m.shape[1] // 8, 8).amax(-1)
               for m, f, least in ((x, xf, 2.0 ** -6), (w, wf, 1.0))]
        acc = acc + 7 * 2.0 ** -13 * (top[0] @ top[1].t())
    if y0 is not None:
        acc = acc + 2.0 ** -24 * (y0.double().abs() + mag)
    return acc + (2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24) * (want.abs() + acc)


@pytest.mark.parametrize("bits,dtype,T,k,n,tile,parts", mx_plans.PRODUCTS)
def test_every_kernel(bits, dtype, T, k, n, tile, parts):
    g = torch.Generator(device="cuda").manual_seed(T + k + n)
    dt = TYPES[dtype]
    x, xv, xf = _rows(bits, T, k, g)
    wc, ws, wv, wf = _codes4(n, k, g)
    w = lb.MxWeight(wc, ws, n, k)
    want = xv @ wv.t()
    got = lb.lora_base_product_mx(x, w, dtype=dt)
    assert bool(((got.double() - want).abs() <= _bound(xv, wv, xf, wf, want, dt, bits, parts=parts)).all())
    y0 = (100 * torch.randn(T, n, generator=g, device="cuda")).to(dt)
    got = lb.lora_base_product_mx(x, w, y=y0.clone(), accumulate=True)
    want = want + y0.double()
    assert bool(((got.double() - want).abs() <= _bound(xv, wv, xf, wf, want, dt, bits, y0, parts)).all())


@pytest.mark.parametrize("bits,dtype,T,E,k,n,tile", mx_plans.EXPERTS)
def test_every_kernel_of_the_experts(bits, dtype, T, E, k, n, tile):
    g = torch.Generator(device="cuda").manual_seed(T + k + n)
    dt = TYPES[dtype]
    ids = mh.random_choices(T, 1, E, T, drop=0.05, skew=1.0)
    seg = lb.lora_expert_segments(torch.from_numpy(ids).cuda(), E)
    off, perm, _ = mh.sort_choices(ids, E)
    x, xv, xf = _rows(bits, T, k, g)
    wc, ws, wv, wf = _codes4(E * n, k, g)
    y0 = (100 * torch.randn(T, n, generator=g, device="cuda")).to(dt)
    w = lb.MxWeight(wc, ws, n, k, experts=E)
    for add in (False, True):
        got = lb.lora_expert_product_mx(x, w, seg, y=y0.clone(), accumulate=add)
        for e in range(E):
            a, b, r = int(off[e]), int(off[e + 1]), slice(e * n, (e + 1) * n)
            old = y0[a:b] if add else None
            want = xv[a:b] @ wv[r].t() + (old.double() if add else 0)
            assert bool(((got[a:b].double() - want).abs() <= _bound(xv[a:b], wv[r], xf[a:b], wf[r], want, dt, bits, old)).all()), (e, add)
        assert torch.equal(got[len(perm):], y0[len(perm):])


@pytest.mark.parametrize("T", [3, 40, 300])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", TYPES)
def test_cancelling_outliers_keep_the_bound(dtype, bits, T):
    """Groups of 8 columns in pairs, one with a product as large as can be that the other cancels, beside codes of every
    size: fp32 y and 4-bit rows lose nothing to the cut."""
    dt = TYPES[dtype]
    rng = np.random.default_rng(T)
    n, k = 136, 512
    wc = rng.integers(0, 16, size=(n, k)).astype(np.uint8)
    xc = (rng.integers(0, 127, size=(T, k)) | rng.integers(0, 2, size=(T, k)) << 7).astype(np.uint8) if bits == 8 else \
        rng.integers(0, 16, size=(T, k)).astype(np.uint8)
    big, sign = (126, 128) if bits == 8 else (7, 8)
    xc[:, 0::16], xc[:, 8::16] = big, big | sign  # +x and -x, against 6 and 6
    wc[:, 0::16] = wc[:, 8::16] = 7
    w = lb.MxWeight(torch.from_numpy(mh.pack(wc)).cuda(), torch.full((n, k // 32), 127, dtype=torch.uint8).cuda(), n, k)
    wv = torch.from_numpy(mh.E2M1[wc]).cuda()
    if bits == 8:
        x = lb.QuantRows(torch.from_numpy(xc).cuda(), torch.full((T, 4), 127, dtype=torch.uint8).cuda(), k)
        xv = torch.from_numpy(qh.E4M3[xc]).cuda()
    else:
        x = lb.MxRows(torch.from_numpy(mh.pack(xc)).cuda(), torch.full((T, k // 32), 127, dtype=torch.uint8).cuda(), k)
        xv = torch.from_numpy(mh.E2M1[xc]).cuda()
    want = xv @ wv.t()
    one = torch.ones((), device="cuda", dtype=torch.float64)
    got = lb.lora_base_product_mx(x, w, dtype=dt)
    assert bool(((got.double() - want).abs() <= _bound(xv, wv, one, one, want, dt, bits)).all())


def test_offsets_past_32_bits():
    """Rows, outputs and weights whose offsets do not fit 32 bits: the last rows of each."""
    k, n = 256, 8
    free = torch.cuda.mem_get_info()[0]
    T = (1 << 32) // 128 + 200  # 4-bit rows of 128 bytes
    if free < 12 << 30:
        pytest.skip("needs 12 GB")
    g = torch.Generator(device="cuda").manual_seed(1)
    wc, ws, wv, _ = _codes4(n, k, g)
    w = lb.MxWeight(wc, ws, n, k)
    codes, scales = torch.zeros(T, 128, dtype=torch.uint8, device="cuda"), torch.full((T, 8), 127, dtype=torch.uint8, device="cuda")
    tail = 70
    c, s, v, _ = _codes4(tail, k, g)
    codes[-tail:], scales[-tail:] = c, s
    x = lb.MxRows(codes, scales, k)
    y = lb.lora_base_product_mx(x, w, dtype=torch.float32)
    want = v @ wv.t()
    assert torch.allclose(y[-tail:].double(), want, rtol=1e-5, atol=1e-5 * float(want.abs().max())) and not y[: T - tail : 1001].any()
    back = lb.lora_dequant_rows_mx(x[T - tail:], torch.float32)
    assert torch.equal(back.double(), v)
    # the same rows as the weight of many outputs
    z = lb.lora_base_product_mx(lb.MxRows(wc, ws, k), x.as_weight(), dtype=torch.float32)
    assert torch.allclose(z[:, -tail:].double(), wv @ v.t(), rtol=1e-5, atol=1e-5 * float(want.abs().max()))
    del z, y
    # and as one expert behind others, the rows of that expert behind the others'
    E = T // 8
    seg = lb.lora_expert_segments(torch.full((300, 1), E - 1, dtype=torch.int32, device="cuda"), E)
    xr, xv, _ = _rows(4, 300, k, g)
    o = lb.lora_expert_product_mx(xr, x.as_weight(E), seg, dtype=torch.float32)
    want = xv @ v[-8:].t() if T % 8 == 0 else None
    if want is not None:
        assert torch.allclose(o.double(), want, rtol=1e-5, atol=1e-5 * float(want.abs().max()))


def test_rows_of_experts_past_32_bits():
    T, d, k = 70000, 8192, 4  # 280000 rows of 16 KB
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    ids = torch.randint(0, 5, (T, k), dtype=torch.int32, device="cuda")
    seg = lb.lora_expert_segments(ids, 5)
    x = torch.randn(T, d, device="cuda").to(torch.bfloat16)
    y = lb.lora_expert_gather(x, seg)
    at = torch.randint(0, T * k, (50,), device="cuda").tolist() + [0, T * k - 1]
    perm = seg.perm.long()
    for i in at:
        assert torch.equal(y[i], x[perm[i] // k])
    w = torch.full((T, k), 0.25, device="cuda")
    assert torch.equal(lb.lora_expert_combine(y, w, seg), x)  # four quarters of a row
    d_o, dw = lb.lora_expert_combine_backward(x, y, w, seg, d_o=y)
    assert torch.equal(d_o[T * k - 1], (0.25 * x[perm[T * k - 1] // k].float()).to(torch.bfloat16))
    assert torch.allclose(dw[-1], x[-1].float().square().sum().expand(k), rtol=1e-4)


def test_two_graphs_share_a_workspace():
    """A workspace is free again when its call is done: two captured calls over one, replayed in turn."""
    g = torch.Generator(device="cuda").manual_seed(5)
    outs, graphs, wants = [], [], []
    ws = torch.empty(lb.LORA_BASE_PRODUCT_MAX_WORKSPACE, dtype=torch.uint8, device="cuda")
    for T, k, n in ((18, 18472, 8), (65, 5656, 8568)):  # k in parts
        x, _, _ = _rows(4, T, k, g)
        wc, s, _, _ = _codes4(n, k, g)
        w = lb.MxWeight(wc, s, n, k)
        y = torch.zeros(T, n, device="cuda")
        wants.append(lb.lora_base_product_mx(x, w, dtype=torch.float32, ws=ws).clone())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lb.lora_base_product_mx(x, w, y=y, ws=ws)
        outs.append((x, w, y))
        graphs.append(graph)
    for _ in range(4):
        for (x, w, y), graph, want in zip(outs, graphs, wants):
            y.fill_(7)
            graph.replay()
        torch.cuda.synchronize()
        for (x, w, y), want in zip(outs, wants):
            assert torch.equal(y, want)
            assert torch.equal(lb.lora_base_product_mx(x, w, dtype=torch.float32, ws=ws), want)  # eager work between


def test_workspaces_of_the_caller_and_their_refusal():
    g = torch.Generator(device="cuda").manual_seed(6)
    x, _, _ = _rows(8, 300, 57344, g)
    wc, s, _, _ = _codes4(136, 57344, g)
    w = lb.MxWeight(wc, s, 136, 57344)
    need = lb.lora_base_product_mx_workspace_bytes(300, 57344, 136)
    assert need > 16
    want = lb.lora_base_product_mx(x, w)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")  # (its contents do not matter)
    assert torch.equal(lb.lora_base_product_mx(x, w, ws=ws[:need]), want)
    assert (ws[need:] == 255).all()
    for bad in (ws[:16], ws[8:need + 8]):
        with pytest.raises(lb.LoraError):
            lb.lora_base_product_mx(x, w, ws=bad)
    with pytest.raises(ValueError):
        lb.lora_base_product_mx(x, w, ws=torch.empty(need, dtype=torch.uint8))
