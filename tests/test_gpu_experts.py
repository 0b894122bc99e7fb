"""Rows to the experts and back, the gradients, and the experts' products, on the GPU against the 64-bit oracle
(mx_helpers).  What only moves rows is exact; sums are held to bounds by their lengths."""
import numpy as np
import pytest
import torch

import mx_helpers as mh
import quant_helpers as qh

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expand_token_adapter_amd as lb

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _batch(T, k, E, seed, drop=0.1, skew=1.0):
    ids = mh.random_choices(T, k, E, seed, drop, skew)
    return ids, lb.lora_expert_segments(torch.from_numpy(ids).cuda(), E), mh.sort_choices(ids, E)


def _tensor(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(TYPES[dtype])


# (tokens, k, experts, columns)
SIZES = [(1, 1, 1, 8), (1, 8, 64, 4096), (7, 3, 5, 264), (33, 2, 8, 1160), (211, 4, 12, 512), (300, 9, 16, 520), (64, 13, 13, 72),
         (1000, 2, 320, 136)]


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (5, 2, 3), (100, 8, 64), (1024, 4, 7), (1025, 4, 7), (3000, 4, 300), (5000, 1, 1024),
                                   (9000, 8, 16), (5003, 1, 1), (140001, 2, 33), (700, 2, 1500), (40000, 2, 1100)])
def test_segments_and_places(T, k, E):
    """Every build (one workgroup, two kernels, three kernels), with dropped choices and ids outside the table."""
    ids = mh.random_choices(T, k, E, T + E)
    if T > 4:
        ids[3, 0], ids[4, -1] = E, -7
    seg = lb.lora_expert_segments(torch.from_numpy(ids).cuda(), E)
    off, perm, pos = mh.sort_choices(ids, E)
    assert np.array_equal(seg.offsets.cpu().numpy(), off)
    assert np.array_equal(seg.perm.cpu().numpy()[: len(perm)], perm)
    assert np.array_equal(seg.pos.cpu().numpy(), pos)
    assert int(seg.err.item()) == (2 if T > 4 else 0)
    plain = lb.lora_segments_build(torch.from_numpy(ids.reshape(-1).copy()).cuda(), E)
    for name in ("counts", "offsets", "sched", "err"):
        assert torch.equal(getattr(seg, name), getattr(plain, name))
    again = lb.lora_expert_segments(torch.full((T, k), -1, dtype=torch.int32, device="cuda"), E, out=seg)
    assert again is seg and (seg.pos == -1).all() and (seg.offsets == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,d", SIZES)
def test_gather_and_its_gradient(T, k, E, d, dtype):
    ids, seg, (off, perm, pos) = _batch(T, k, E, T + d)
    x = _tensor((T, d), dtype, 1)
    y = torch.full((T * k, d), 9.0, dtype=TYPES[dtype], device="cuda")
    lb.lora_expert_gather(x.cuda(), seg, y=y)
    n = len(perm)
    assert torch.equal(y[:n].cpu(), x[torch.from_numpy(perm // k)])
    assert (y[n:] == 9).all()  # rows behind the last expert's
    dy = _tensor((T * k, d), dtype, 2)
    dy[n:] = float("nan")  # and they are not read
    rows = _f64(dy)
    want = np.zeros((T, d))
    mag = np.zeros((T, d))
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                want[t] += rows[pos[t, j]]
                mag[t] += np.abs(rows[pos[t, j]])
    got = lb.lora_expert_gather_backward(dy.cuda(), seg)
    bound = lambda v, m: k * 2.0 ** -24 * m + HALF[dtype] * (np.abs(v) + k * 2.0 ** -24 * m)
    assert np.all(np.abs(_f64(got) - want) <= bound(want, mag))
    dx = _tensor((T, d), dtype, 3)
    got = lb.lora_expert_gather_backward(dy.cuda(), seg, dx=dx.cuda(), accumulate=True)
    total = want + _f64(dx)
    assert np.all(np.abs(_f64(got) - total) <= bound(total, 2 * (mag + np.abs(_f64(dx)))))
    # the gradient is the gather's: <gather(x), dy> = <x, gather_backward(dy)>
    lhs = (_f64(y)[:n] * rows[:n]).sum()
    assert abs(lhs - (_f64(x) * want).sum()) <= 1e-9 * (np.abs(_f64(y)[:n] * rows[:n]).sum() + 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,d", SIZES)
def test_combine_and_its_gradient(T, k, E, d, dtype):
    ids, seg, (off, perm, pos) = _batch(T, k, E, T + d + 1)
    n = len(perm)
    o = _tensor((T * k, d), dtype, 1)
    o[n:] = float("nan")
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(2))
    w[torch.from_numpy(pos) < 0] = float("nan")  # a choice without a place adds nothing, whatever its weight
    dy = _tensor((T, d), dtype, 3)
    ov, wv, dyv = _f64(o), _f64(w), _f64(dy)
    want, mag, dw, dmag = np.zeros((T, d)), np.zeros((T, d)), np.zeros((T, k)), np.zeros((T, k))
    d_o = np.full((T * k, d), 9.0)
    for t in range(T):
        for j in range(k):
            p = pos[t, j]
            if p >= 0:
                want[t] += wv[t, j] * ov[p]
                mag[t] += np.abs(wv[t, j] * ov[p])
                dw[t, j] = (dyv[t] * ov[p]).sum()
                dmag[t, j] = np.abs(dyv[t] * ov[p]).sum()
                d_o[p] = wv[t, j] * dyv[t]
    got = lb.lora_expert_combine(o.cuda(), w.cuda(), seg)
    bound = lambda v, m: (k + 1) * 2.0 ** -24 * m + HALF[dtype] * (np.abs(v) + (k + 1) * 2.0 ** -24 * m)
    assert np.all(np.abs(_f64(got) - want) <= bound(want, mag))
    y = _tensor((T, d), dtype, 4)
    got = lb.lora_expert_combine(o.cuda(), w.cuda(), seg, y=y.cuda(), accumulate=True)
    assert np.all(np.abs(_f64(got) - want - _f64(y)) <= bound(want + _f64(y), 2 * (mag + np.abs(_f64(y)))))
    out = torch.full((T * k, d), 9.0, dtype=TYPES[dtype], device="cuda")
    g_o, g_w = lb.lora_expert_combine_backward(dy.cuda(), o.cuda(), w.cuda(), seg, d_o=out)
    assert g_o is out and g_w.dtype == torch.float32
    assert np.all(np.abs(_f64(g_o) - d_o) <= (HALF[dtype] + 2.0 ** -24) * np.abs(d_o)) and (out[n:] == 9).all()
    # a lane adds its columns (at most d / 64 of them), then 6 steps over the wave and 3 over the waves
    assert np.all(np.abs(_f64(g_w) - dw) <= (d / 64 + 8 + 9) * 2.0 ** -24 * dmag)
    again = lb.lora_expert_combine_backward(dy.cuda(), o.cuda(), w.cuda(), seg)
    assert torch.equal(again[0][:n], g_o[:n]) and torch.equal(again[1], g_w) and (again[0][n:] == 0).all()
    # in place: the rows' gradient over the rows
    same = o.cuda()
    in_place, dw_in_place = lb.lora_expert_combine_backward(dy.cuda(), same, w.cuda(), seg, d_o=same)
    assert torch.equal(in_place[:n], g_o[:n]) and torch.equal(dw_in_place, g_w)


def test_combine_gradient_by_differences():
    """dw and d_o against differences of the combine itself (fp32: the function is linear in each)."""
    T, k, E, d = 9, 3, 4, 72
    ids, seg, (off, perm, pos) = _batch(T, k, E, 5)
    o, w, dy = (_tensor(s, "f32", i).cuda() for i, s in enumerate([(T * k, d), (T, k), (T, d)]))
    f = lambda o, w: float((lb.lora_expert_combine(o, w, seg).double() * dy.double()).sum())
    d_o, dw = lb.lora_expert_combine_backward(dy, o, w, seg)
    base = f(o, w)
    for t, j in ((0, 0), (4, 2), (8, 1)):
        w2 = w.clone()
        w2[t, j] += 1.0
        assert abs(f(o, w2) - base - float(dw[t, j])) <= 1e-3  # (sums of 648 products of order 1, each to 2^-22)
    for p, c in ((0, 0), (len(perm) - 1, 71), (3, 10)):
        o2 = o.clone()
        o2[p, c] += 1.0
        assert abs(f(o2, w) - base - float(d_o[p, c])) <= 1e-3


def test_pitches_and_places_outside_the_rows():
    T, k, E, d = 40, 3, 6, 136
    ids, seg, (off, perm, pos) = _batch(T, k, E, 8)
    wide = torch.full((T, d + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :d] = _tensor((T, d), "bf16", 1)
    x = wide[:, :d].contiguous()
    out = torch.full((T * k, d + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    lb.lora_expert_gather(wide[:, :d], seg, y=out[:, :d])
    rows = lb.lora_expert_gather(x, seg)
    n = len(perm)
    assert torch.equal(out[:n, :d], rows[:n]) and (out[:, d:] == 5).all() and (out[n:] == 5).all()
    w = torch.rand(T, k, device="cuda")
    y = torch.full((T, d + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    lb.lora_expert_combine(out[:, :d], w, seg, y=y[:, :d])
    assert torch.equal(y[:, :d], lb.lora_expert_combine(rows, w, seg)) and (y[:, d:] == 5).all()
    a = lb.lora_expert_combine_backward(wide[:, :d], out[:, :d], w, seg)
    b = lb.lora_expert_combine_backward(x, rows, w, seg)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # places that no build gives count as none
    seg.pos[0, 0], seg.pos[1, 1] = T * k, -5
    before = out.clone()
    lb.lora_expert_gather(x, seg, y=out[:, :d])
    assert torch.equal(out, before)
    seg.pos[0, 0] = seg.pos[1, 1] = -1
    want = lb.lora_expert_combine(rows, w, seg)
    seg.pos[0, 0], seg.pos[1, 1] = 2 ** 31 - 1, -2 ** 31
    assert torch.equal(lb.lora_expert_combine(rows, w, seg), want)


# ------------------------------------------------------------------ products

PRODUCTS = [(1, 1, 1, 264, 40), (1, 8, 64, 520, 136), (3, 2, 4, 4096, 72), (40, 4, 32, 1160, 264), (150, 2, 8, 520, 1032),
            (700, 2, 4, 1032, 520), (2000, 1, 3, 392, 776), (300, 3, 100, 264, 136), (1500, 4, 6, 264, 1288)]


def _weights(E, n, k, g):
    c, s = mh.random_mx(E * n, k, g, scale=0.02)
    return lb.MxWeight(c.cuda(), s.cuda(), n, k, experts=E), mh.values(mh.unpack(c.numpy()), s.numpy(), k).reshape(E, n, k), \
        mh.expand(s.numpy(), 32, k).reshape(E, n, k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,top,E,k,n", PRODUCTS)
def test_expert_product(T, top, E, k, n, bits, dtype):
    g = torch.Generator().manual_seed(T + k)
    ids, seg, (off, perm, _) = _batch(T, top, E, T + n, drop=0.15, skew=1.5)
    R = T * top
    w, wv, wf = _weights(E, n, k, g)
    if bits == 4:
        xc, xs = mh.random_mx(R, k, g)
        x, xv, xf = lb.MxRows(xc.cuda(), xs.cuda(), k), mh.values(mh.unpack(xc.numpy()), xs.numpy(), k), mh.expand(xs.numpy(), 32, k)
    else:
        xc, xs = mh.random_rows8(R, k, g)
        nb = -(-k // 128)
        x, xv, xf = lb.QuantRows(xc.cuda(), xs.cuda(), k), qh.values(xc.numpy(), xs.numpy()[:, :nb], k), mh.expand(xs.numpy()[:, :nb], 128, k)
    x.scales[len(perm):] = 255  # rows of no expert are not read
    dt = TYPES[dtype]
    y0 = _tensor((R, n), dtype, 6)
    plain = torch.full((R, n), 9.0, dtype=dt, device="cuda")
    lb.lora_expert_product_mx(x, w, seg, y=plain)
    added = lb.lora_expert_product_mx(x, w, seg, y=y0.cuda(), accumulate=True)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a == b:
            continue
        want = xv[a:b] @ wv[e].T
        off_by = np.abs(_f64(plain)[a:b] - want)
        assert np.all(off_by <= mh.product_bound(xv[a:b], wv[e], want, dt, bits, wf[e], xf[a:b])), (e, off_by.max())
        old = _f64(y0)[a:b]
        off_by = np.abs(_f64(added)[a:b] - want - old)
        assert np.all(off_by <= mh.product_bound(xv[a:b], wv[e], want + old, dt, bits, wf[e], xf[a:b], old)), (e, off_by.max())
    rest = int(off[E])
    assert (plain[rest:] == 9).all() and torch.equal(added[rest:].cpu(), y0[rest:])
    assert torch.equal(lb.lora_expert_product_mx(x, w, seg, dtype=dt)[:rest], plain[:rest])


@pytest.mark.parametrize("bits", [4, 8])
def test_one_expert_with_every_row_and_none_with_any(bits):
    g = torch.Generator().manual_seed(3)
    T, k, n, E = 300, 264, 136, 5
    w, wv, wf = _weights(E, n, k, g)
    x = lb.lora_quant_rows_mx(torch.randn(T, k, generator=g).cuda()) if bits == 4 else lb.lora_quant_rows(torch.randn(T, k, generator=g).cuda())
    ids = torch.full((T, 1), 3, dtype=torch.int32, device="cuda")
    seg = lb.lora_expert_segments(ids, E)
    y = lb.lora_expert_product_mx(x, w, seg, dtype=torch.float32)
    one = lb.MxWeight(w.codes[3 * n : 4 * n], w.scales[3 * n : 4 * n], n, k)
    want = lb.lora_base_product_mx(x, one, dtype=torch.float32)
    assert torch.allclose(y, want, rtol=0, atol=float(want.abs().max()) * 2.0 ** -17)  # (another split of k)
    lb.lora_expert_segments(torch.full_like(ids, -1), E, out=seg)
    z = torch.full((T, n), 9.0, device="cuda")
    assert (lb.lora_expert_product_mx(x, w, seg, y=z) == 9).all()


def test_the_binding_checks_its_arguments():
    ids, seg, _ = _batch(10, 2, 4, 1)
    x = torch.zeros(10, 64, device="cuda")
    rows = torch.zeros(20, 64, device="cuda")
    w = torch.zeros(10, 2, device="cuda")
    for call in (lambda: lb.lora_expert_gather(rows, seg), lambda: lb.lora_expert_gather(x, seg, y=x),
                 lambda: lb.lora_expert_gather(x, seg, y=rows.bfloat16()), lambda: lb.lora_expert_gather_backward(x, seg),
                 lambda: lb.lora_expert_gather_backward(rows, seg, accumulate=True),
                 lambda: lb.lora_expert_combine(rows, w.double(), seg), lambda: lb.lora_expert_combine(rows, w[:, :1], seg),
                 lambda: lb.lora_expert_combine_backward(x, rows[:, :32], w, seg),
                 lambda: lb.lora_expert_combine_backward(x, rows, w, seg, dw=w.bfloat16()),
                 lambda: lb.lora_expert_segments(torch.zeros(3, 2, dtype=torch.int32, device="cuda"), 4, out=seg)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lb.lora_expert_gather(x, lb.lora_segments_build(torch.zeros(10, dtype=torch.int32, device="cuda"), 4)),
                 lambda: lb.lora_expert_gather(x.half(), seg, y=rows.half())):
        with pytest.raises(TypeError):
            call()
    q = lb.lora_quant_rows_mx(rows)
    weight = lb.lora_quant_weight_mx(torch.zeros(4, 8, 64, device="cuda"))
    with pytest.raises(ValueError):
        lb.lora_expert_product_mx(q[:10], weight, seg)
    with pytest.raises(ValueError):
        lb.lora_expert_product_mx(q, lb.lora_quant_weight_mx(torch.zeros(3, 8, 64, device="cuda")), seg)
    with pytest.raises(ValueError):
        lb.lora_base_product_mx(q, weight)
    empty = lb.lora_expert_segments(torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 4)
    assert lb.lora_expert_gather(x[:0], empty).shape == (0, 64) and lb.lora_expert_combine(rows[:0], w[:0], empty).shape == (0, 64)
