"""The 8-bit calls where they can go wrong: entries and rows that the backward has to
leave out on each of its routes, pitches at their limit, offsets past 32 bits, and
two captured graphs over one workspace."""
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

# ranks, d_in, d_out, rows: the streaming backward, the two-pass one, the one with 256-column tiles
ROUTES = {"stream": ([16, 5, 20, 12], 264, 1032, 299), "two-pass": ([64, 40, 72, 8], 264, 520, 299),
          "wide": ([64, 40, 72, 8], 2056, 4104, 2600)}


def _case(route, dtype="bf16"):
    """Four adapters and rows without one; the third's rank is above the r_max of the calls."""
    ranks, d_in, d_out, T = ROUTES[route]
    rng = np.random.default_rng(6)
    ids = np.concatenate([np.full(T // 3, 0), rng.integers(-1, 4, size=T // 4),
                          np.full(T - T // 3 - T // 4, 3)]).astype(np.int32)
    wl = workloads.custom(ids, ranks, d_in, d_out, dtype, seed=6, scales=[2.0, -0.5, 1.5, 1.0], ft_start=0, ft_count=T,
                          name="quant-edges")
    return GpuCase(wl), (16 if route == "stream" else 64)


class _Run:
    """Outputs of one backward, filled with ones before."""

    def __init__(self, c, r_max, x, dy, none=(), fn=None, ids=None, pad=0):
        wl, dev = c.wl, c.dev
        self.dA = [torch.ones(a.shape, device=dev) for a in wl.A]
        self.dB = [torch.ones(b.shape, device=dev) for b in wl.B]
        grads = lb.GradTable([None if i in none else t for i, t in enumerate(self.dA)],
                             [None if i in none else t for i, t in enumerate(self.dB)])
        self.wide = torch.ones(wl.T, wl.d_in + pad, dtype=c.x.dtype, device=dev)
        self.dx = self.wide[:, :wl.d_in]
        seg = lb.lora_segments_build(c.ids if ids is None else ids, wl.num_adapters)
        (fn or lb.lora_backward_quant)(x, dy, c.table, grads, seg, dx=self.dx, r_max=r_max)
        torch.cuda.synchronize()
        self.err = int(seg.err.item())

    def tensors(self):
        return self.dA + self.dB + [self.dx]


@pytest.mark.parametrize("route", ROUTES)
def test_bad_and_missing_entries(route):
    """Adapter 2 is above r_max and adapter 1 has no gradients: neither is written, both are counted, the others
    are as if alone."""
    c, r_max = _case(route)
    wl = c.wl
    q, dy = lb.lora_quant_rows(c.x), to_dev(wl.dy, "bf16", c.dev)
    got = _Run(c, r_max, q, dy, none=(1,))
    old = _Run(c, r_max, lb.lora_dequant_rows(q), dy, none=(1,), fn=lb.lora_backward)
    assert got.err == old.err > 0
    assert torch.equal(got.dx, old.dx)  # dX of adapter 1's rows is there, of adapter 2's not
    at = torch.from_numpy(wl.ids == 2).cuda()
    assert (got.dx[at] == 1).all() and all((t[i] == 1).all() for t in (got.dA, got.dB) for i in (1, 2))
    ids = c.ids.clone()
    ids[(ids == 1) | (ids == 2)] = -1
    alone = _Run(c, r_max, q, dy, ids=ids)
    assert alone.err == 0
    ref = oracle.from_workload(wl)
    xv = qh.values(q.codes.cpu().numpy(), q.scales.cpu().numpy()[:, : -(-wl.d_in // 128)], wl.d_in)
    for a in (0, 3):
        rows = wl.ids == a
        g, v = ref["dy"][rows] @ ref["B"][a], xv[rows] @ ref["A"][a].T
        for t, want in ((got.dA[a], g.T @ xv[rows]), (got.dB[a], ref["dy"][rows].T @ v)):
            assert rel_err(t, 1 + ref["scales"][a] * want) <= TOL["bf16"]
    assert all(rel_err(got.dA[a], alone.dA[a].double().cpu().numpy()) <= 1e-5 for a in (0, 3))


@pytest.mark.parametrize("route", ROUTES)
def test_rows_without_an_adapter_are_not_read_into_a_sum(route):
    """NaN in the saved rows and dY of rows without an adapter, adapters without rows: nothing of them is written."""
    c, r_max = _case(route)
    q, dy = lb.lora_quant_rows(c.x), to_dev(c.wl.dy, "bf16", c.dev)
    ids = c.ids.clone()
    ids[(ids == 2) | (ids == 1)] = -1
    want = _Run(c, r_max, q, dy, ids=ids)
    q.codes[ids < 0] = 0x7F
    q.scales[ids < 0] = 255
    dy[ids < 0] = float("nan")
    got = _Run(c, r_max, q, dy, ids=ids)
    assert got.err == 0 and all(torch.equal(a, b) for a, b in zip(got.tensors(), want.tensors()))
    assert (got.dx[ids < 0] == 1).all() and all((t[i] == 1).all() for t in (got.dA, got.dB) for i in (1, 2))
    none = _Run(c, r_max, q, dy, ids=torch.full_like(ids, -1))  # no row has an adapter
    assert none.err == 0 and all((t == 1).all() for t in none.tensors())


@pytest.mark.parametrize("route", ROUTES)
def test_pitches_of_the_backward(route):
    c, r_max = _case(route)
    wl = c.wl
    q, dy = lb.lora_quant_rows(c.x), to_dev(wl.dy, "bf16", c.dev)
    ids = c.ids.clone()
    ids[ids == 2] = -1
    want = _Run(c, r_max, q, dy, ids=ids)
    nan = dict(dtype=torch.bfloat16, device="cuda")
    wide_dy = torch.full((wl.T, wl.d_out + 24), float("nan"), **nan)
    wide_dy[:, :wl.d_out] = dy
    codes = torch.full((wl.T, q.codes.shape[1] + 128), 0x7F, dtype=torch.uint8, device="cuda")
    scales = torch.full((wl.T, q.scales.shape[1] + 4), 255, dtype=torch.uint8, device="cuda")
    codes[:, : q.codes.shape[1]], scales[:, : q.scales.shape[1]] = q.codes, q.scales
    got = _Run(c, r_max, lb.QuantRows(codes, scales, wl.d_in), wide_dy[:, :wl.d_out], ids=ids, pad=40)
    assert all(torch.equal(a, b) for a, b in zip(got.tensors(), want.tensors()))
    assert (got.wide[:, wl.d_in:] == 1).all()


@pytest.mark.parametrize("dtype,ranks,T", [("f32", [32, 7, 20], 3100), ("bf16", [32, 7, 20], 3100), ("f32", [64, 16, 33], 1600),
                                           ("bf16", [128, 72, 9], 1100), ("f32", [128, 72, 9], 1100)])
def test_wide_tiles_of_every_rank_class(dtype, ranks, T):
    """256-column tiles for r_max to 32, to 64 and to 128, v saved and not, with and without dX, against 64 bits."""
    d_in, d_out = 4104, 4112
    rng = np.random.default_rng(T)
    ids = np.concatenate([np.full(T // 2, 0), rng.integers(-1, 3, size=T // 4), np.full(T - T // 2 - T // 4, 1)])
    wl = workloads.custom(ids.astype(np.int32), ranks, d_in, d_out, dtype, seed=T, scales=[2.0, -0.5, 1.5], ft_start=0, ft_count=T,
                          name="quant-wide")
    c = GpuCase(wl)
    q, dy = lb.lora_quant_rows(c.x), to_dev(wl.dy, dtype, c.dev)
    ref = oracle.from_workload(wl)
    xv = qh.values(q.codes.cpu().numpy(), q.scales.cpu().numpy()[:, : -(-d_in // 128)], d_in)
    dx_ref, dA_ref, dB_ref, _, _ = oracle.backward(xv, ref["dy"], ref["ids"], ref["ranks"], ref["scales"], ref["A"], ref["B"])
    seg = lb.lora_segments_build(c.ids, 3)
    v = lb.lora_shrink(lb.lora_dequant_rows(q, c.x.dtype), c.table, seg)
    for v_saved, with_dx in ((None, True), (v, False)):
        dA, dB = ([torch.zeros(t.shape, device=c.dev) for t in m] for m in (wl.A, wl.B))
        dx = torch.zeros(T, d_in, dtype=c.x.dtype, device=c.dev) if with_dx else None
        lb.lora_backward_quant(q, dy, c.table, lb.GradTable(dA, dB), seg, dx=dx, v_saved=v_saved)
        torch.cuda.synchronize()
        errs = {f"dA{a}": rel_err(dA[a], dA_ref[a]) for a in range(3)} | {f"dB{a}": rel_err(dB[a], dB_ref[a]) for a in range(3)}
        if with_dx:
            errs["dx"] = rel_err(dx, dx_ref)
        assert int(seg.err.item()) == 0 and all(e <= TOL[dtype] for e in errs.values()), errs


def test_two_graphs_over_one_workspace():
    """A product with a split k and a wide backward, captured over the same workspace and replayed in turn."""
    c, r_max = _case("wide")
    wl = c.wl
    ids = c.ids.clone()
    ids[ids == 2] = -1
    q, dy = lb.lora_quant_rows(c.x), to_dev(wl.dy, "bf16", c.dev)
    seg = lb.lora_segments_build(ids, 4)
    xs = lb.lora_quant_rows(torch.randn(64, 14336, device="cuda"))
    w = lb.lora_quant_weight(torch.randn(136, 14336, device="cuda"))
    need = (lb.lora_base_product_workspace_bytes(64, 14336, 136),
            lb.lora_backward_quant_workspace_bytes(torch.bfloat16, wl.T, wl.d_in, wl.d_out, 64))
    ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    y = torch.zeros(64, 136, device="cuda")
    dA, dB = ([torch.zeros(t.shape, device="cuda") for t in m] for m in (wl.A, wl.B))
    grads = lb.GradTable(dA, dB)

    def product():
        lb.lora_base_product(xs, w, y=y, ws=ws)

    def backward():
        for t in dA + dB:
            t.zero_()
        lb.lora_backward_quant(q, dy, c.table, grads, seg, r_max=r_max, ws=ws)

    graphs = []
    for f in (product, backward):
        f()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for k in range(3):
        xs.codes.copy_(lb.lora_quant_rows(torch.randn(64, 14336, device="cuda") + k).codes)
        dy.copy_(torch.randn(dy.shape, device="cuda"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in [y] + dA + dB]
        product()
        backward()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, [y] + dA + dB)), k


def test_base_product_at_the_largest_pitch():
    """Rows 2^22 bytes apart, the limit: 300 rows of x and 264 of W, more than a tile of each."""
    g = torch.Generator().manual_seed(3)
    x = lb.lora_quant_rows(torch.randn(300, 392, generator=g).cuda())
    w = lb.lora_quant_weight(torch.randn(264, 392, generator=g).cuda())
    want = lb.lora_base_product(x, w)
    far = []
    for q in (x, w):
        codes = torch.empty(q.codes.shape[0], 1 << 22, dtype=torch.uint8, device="cuda")
        codes[:, :512] = q.codes
        far.append(codes)
    got = lb.lora_base_product(lb.QuantRows(far[0], x.scales, 392), lb.QuantWeight(far[1], w.scales, 264, 392))
    assert torch.equal(got, want)
    codes = torch.empty(2, (1 << 22) + 128, dtype=torch.uint8, device="cuda")
    with pytest.raises(lb.LoraError):
        lb.lora_base_product(lb.QuantRows(codes, x.scales[:2], 392), w)


def test_offsets_past_32_bits():
    """450000 rows of 5120: 2.3 GB of codes, 4.6 GB of bf16; rows on both sides of 2^31 bytes and the last ones."""
    T, d, n, r = 450000, 5120, 16, 16
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    rows = torch.cat([torch.arange(40), 2 ** 31 // (2 * d) + torch.arange(-20, 20), 2 ** 31 // d + torch.arange(-20, 20),
                      T - 40 + torch.arange(40)])
    at = rows.cuda()
    q = lb.lora_quant_rows(x)
    codes, scales = q.codes[at].cpu().numpy(), q.scales[at].cpu().numpy()
    want_codes, want_scales = qh.quant(x[at].cpu().double().numpy())
    assert np.array_equal(codes, want_codes) and np.array_equal(scales, want_scales)
    xv = qh.values(codes, scales, d)
    x.zero_()
    lb.lora_dequant_rows(q, out=x)
    assert np.array_equal(x[at].cpu().double().numpy(), xv)
    del x
    w = lb.lora_quant_weight(0.02 * torch.randn(n, d, device="cuda", generator=gen))
    wv = qh.values(w.codes.cpu().numpy(), w.scales.cpu().numpy(), d, 128)
    for dt in (torch.bfloat16, torch.float32):
        y = lb.lora_base_product(q, w, dtype=dt)[at].cpu().double().numpy()
        assert (np.abs(y - xv @ wv.T) <= qh.base_bound(xv, wv, xv @ wv.T, dt)).all()
    # the backward of the same rows, two adapters; every other row has none
    A = [(0.02 * torch.randn(r, d, device="cuda", generator=gen)).bfloat16() for _ in range(2)]
    B = [(0.02 * torch.randn(n, r, device="cuda", generator=gen)).bfloat16() for _ in range(2)]
    table = lb.AdapterTable(A, B, [1.0, 2.0])
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    ids[at] = torch.arange(len(rows), device="cuda", dtype=torch.int32) % 2
    dy = torch.randn(T, n, device="cuda", generator=gen).bfloat16()
    dA, dB = [torch.zeros(r, d, device="cuda") for _ in A], [torch.zeros(n, r, device="cuda") for _ in B]
    seg = lb.lora_segments_build(ids, 2)
    lb.lora_backward_quant(q, dy, table, lb.GradTable(dA, dB), seg)
    torch.cuda.synchronize()
    assert int(seg.err.item()) == 0
    dyv, idv = dy[at].cpu().double().numpy(), ids[at].cpu().numpy()
    for a, s in ((0, 1.0), (1, 2.0)):
        m = idv == a
        Av, Bv = A[a].cpu().double().numpy(), B[a].cpu().double().numpy()
        assert rel_err(dA[a], s * (dyv[m] @ Bv).T @ xv[m]) <= TOL["bf16"]
        assert rel_err(dB[a], s * dyv[m].T @ (xv[m] @ Av.T)) <= TOL["bf16"]


def test_refusals_of_types():
    x, w = lb.lora_quant_rows(torch.randn(4, 256, device="cuda")), lb.lora_quant_weight(torch.randn(16, 256, device="cuda"))
    plain = torch.randn(4, 256, device="cuda")
    for f in (lambda: lb.lora_quant_rows(plain, out=w), lambda: lb.lora_quant_weight(plain, out=x),
              lambda: lb.lora_dequant_rows(w), lambda: lb.lora_base_product(w, x), lambda: lb.lora_base_product(plain, w),
              lambda: lb.lora_backward_quant(plain, None, None, None, None)):
        with pytest.raises(TypeError):
            f()
