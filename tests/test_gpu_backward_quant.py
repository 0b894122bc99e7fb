"""lora_backward_quant: the adapter backward from saved 8-bit rows.

A restored value has 4 significant bits, so it is a bf16 number and the
backward from the codes is lora_backward on the restored rows: dX bit for bit,
dA and dB but for g's and v's bits beyond 16 and the order of the fp32 sums.  It
is also held to the formulas in 64 bits and to differences."""
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


def _wl(dtype, ranks, d_in, d_out, T=299, seed=5, none=True):
    rng = np.random.default_rng(seed)
    A = len(ranks)
    ids = np.concatenate([np.full(T // 3, A - 1), rng.integers(-1 if none else 0, A, size=T // 6),
                          np.full(T - T // 3 - T // 6, 0)]).astype(np.int32)
    return workloads.custom(ids, ranks, d_in, d_out, dtype, seed=seed, name="quant-bwd",
                            scales=[2.0, -0.5, 1.5, 3.0, 1.0, 0.25][:A], ft_start=0, ft_count=T)


def _run(c, x, fn, v=None, with_dx=True, init=False):
    wl, dev = c.wl, c.dev
    g = torch.Generator().manual_seed(2)
    fill = (lambda s, dt: torch.randn(s, generator=g).to(dt).to(dev)) if init else (lambda s, dt: torch.zeros(s, dtype=dt, device=dev))
    dA = [fill(a.shape, torch.float32) for a in wl.A]
    dB = [fill(b.shape, torch.float32) for b in wl.B]
    dx = fill((wl.T, wl.d_in), c.x.dtype) if with_dx else None
    seg = lb.lora_segments_build(c.ids, wl.num_adapters)
    fn(x, to_dev(wl.dy, wl.dtype, dev), c.table, lb.GradTable(dA, dB), seg, dx=dx, v_saved=v)
    torch.cuda.synchronize()
    assert int(seg.err.item()) == 0
    return dA + dB + ([dx] if with_dx else [])


CASES = [("bf16", [16, 5, 12, 1], 264, 1032), ("bf16", [16], 520, 392), ("bf16", [64, 24, 8], 392, 264),
         ("bf16", [128, 40], 136, 520), ("f32", [16, 5, 12], 264, 136), ("f32", [64, 33], 136, 264)]


def _same_as_restored(c, got, want, x):
    """got (from the codes) against want (lora_backward on the restored rows x): dX equal, dA and dB within
    what g and v in 18 bits and two orders of the fp32 sums may differ by."""
    wl = c.wl
    n = wl.num_adapters
    assert all(torch.equal(a, b) for a, b in zip(got[2 * n:], want[2 * n:]))  # dX
    ref = oracle.from_workload(wl)
    xv = x.double().cpu().numpy()
    # each sum runs over the adapter's rows (products exact or with g, v in 18 bits), at most rows + 64
    # additions deep, each off by 2^-23 of the magnitudes at most; then s times it is added to what is there
    for a in range(n):
        at = wl.ids == a
        dy = ref["dy"][at]
        g, v = dy @ ref["B"][a], xv[at] @ ref["A"][a].T
        for k, mag in ((a, np.abs(g).T @ np.abs(xv[at])), (n + a, np.abs(dy).T @ np.abs(v))):
            tol = (2 * (at.sum() + 64) * 2.0 ** -23 + 2.0 ** -18) * abs(ref["scales"][a]) * mag
            tol = tol + 2.0 ** -22 * (np.abs(want[k].double().cpu().numpy()) + mag * abs(ref["scales"][a]))
            off = np.abs(got[k].double().cpu().numpy() - want[k].double().cpu().numpy())
            assert (off <= tol).all(), (k, float((off / np.maximum(tol, 1e-300)).max()))


@pytest.mark.parametrize("save_v", [True, False])
@pytest.mark.parametrize("dtype,ranks,d_in,d_out", CASES)
def test_equals_the_backward_on_restored_rows(dtype, ranks, d_in, d_out, save_v):
    c = GpuCase(_wl(dtype, ranks, d_in, d_out))
    q = lb.lora_quant_rows(c.x)
    restored = lb.lora_dequant_rows(q, c.x.dtype)
    seg = lb.lora_segments_build(c.ids, c.wl.num_adapters)
    v = lb.lora_shrink(restored, c.table, seg) if save_v else None
    for with_dx, init in ((True, True), (False, False)):
        got = _run(c, q, lb.lora_backward_quant, v, with_dx, init)
        want = _run(c, restored, lb.lora_backward, v, with_dx, init)
        _same_as_restored(c, got, want, restored)


# (the first four are wide enough for the 256-column tiles)
@pytest.mark.parametrize("dtype,ranks,d_in,d_out", [("bf16", [8, 128, 33, 64], 2056, 1032), ("bf16", [32, 20, 7, 16], 6152, 6152),
                                                    ("bf16", [64, 33, 8, 48], 2056, 4104), ("f32", [8, 128, 33, 64], 2056, 1032),
                                                    ("bf16", [8, 72, 33, 64], 264, 520), ("f32", [8, 16, 5, 12], 264, 520)])
def test_many_rows_and_cut_tiles(dtype, ranks, d_in, d_out):
    """Long row groups whose tiles are cut between many workgroups, ranks on both sides of a block of 64."""
    rng = np.random.default_rng(4)
    ids = np.concatenate([np.full(1500, 1), rng.integers(-1, 4, size=400), np.full(900, 3)]).astype(np.int32)
    wl = workloads.custom(ids, ranks, d_in, d_out, dtype, seed=4, name="quant-long", scales=[2.0, 1.0, -1.0, 0.5],
                          ft_start=0, ft_count=len(ids))
    c = GpuCase(wl)
    q = lb.lora_quant_rows(c.x)
    restored = lb.lora_dequant_rows(q, c.x.dtype)
    _same_as_restored(c, _run(c, q, lb.lora_backward_quant), _run(c, restored, lb.lora_backward), restored)


@pytest.mark.parametrize("T", [1, 2, 31, 33, 64])
def test_few_rows(T):
    c = GpuCase(_wl("bf16", [16, 8], 136, 264, T=T, none=False))
    q = lb.lora_quant_rows(c.x)
    restored = lb.lora_dequant_rows(q, c.x.dtype)
    _same_as_restored(c, _run(c, q, lb.lora_backward_quant), _run(c, restored, lb.lora_backward), restored)


@pytest.mark.parametrize("dtype,ranks,d_in,d_out", CASES)
def test_against_the_formulas_in_64_bits(dtype, ranks, d_in, d_out):
    c = GpuCase(_wl(dtype, ranks, d_in, d_out, seed=8))
    q = lb.lora_quant_rows(c.x)
    ref = oracle.from_workload(c.wl)
    xv = qh.values(q.codes.cpu().numpy(), q.scales.cpu().numpy()[:, : -(-d_in // 128)], d_in)
    dx, dA, dB, _, _ = oracle.backward(xv, ref["dy"], ref["ids"], ref["ranks"], ref["scales"], ref["A"], ref["B"])
    got = _run(c, q, lb.lora_backward_quant)
    used = sorted(set(int(i) for i in c.wl.ids if i >= 0))
    n = c.wl.num_adapters
    errs = {f"dA{a}": rel_err(got[a], dA[a]) for a in used}
    errs |= {f"dB{a}": rel_err(got[n + a], dB[a]) for a in used}
    errs["dx"] = rel_err(got[-1], dx)
    assert all(e <= TOL[dtype] for e in errs.values()), errs


def test_against_differences():
    """L = sum dy * s B (A x) is linear in each of A, B and x: a central difference along a direction is exact."""
    c = GpuCase(_wl("f32", [16, 5], 136, 264, none=False))
    wl = c.wl
    q = lb.lora_quant_rows(c.x)
    xv = qh.values(q.codes.cpu().numpy(), q.scales.cpu().numpy()[:, :2], 136)
    got = [g.double().cpu().numpy() for g in _run(c, q, lb.lora_backward_quant)]
    ref = oracle.from_workload(wl)

    def loss(A, B, x):
        y = np.zeros((wl.T, wl.d_out))
        for a in range(wl.num_adapters):
            at = wl.ids == a
            y[at] = ref["scales"][a] * (x[at] @ A[a].T) @ B[a].T
        return float((ref["dy"] * y).sum())

    rng = np.random.default_rng(1)
    for k in range(2 * wl.num_adapters + 1):
        A, B, x = [m.copy() for m in ref["A"]], [m.copy() for m in ref["B"]], xv.copy()
        at = A[k] if k < 2 else B[k - 2] if k < 4 else x
        e = rng.standard_normal(at.shape)
        h = 0.5
        at += h * e
        up = loss(A, B, x)
        at -= 2 * h * e
        diff = (up - loss(A, B, x)) / (2 * h)
        # each gradient element is within 1e-5 of the largest (the fp32 bar of every backward test)
        assert abs(float((got[k] * e).sum()) - diff) <= 1e-5 * np.abs(got[k]).max() * np.abs(e).sum()


def test_a_slice_of_a_longer_checkpoint():
    """Fine-tuning rows in the middle of a checkpoint with a wider pitch, whose other rows are NaN."""
    c = GpuCase(_wl("bf16", [16, 8], 264, 520))
    T = c.wl.T
    q = lb.lora_quant_rows(c.x)
    codes = torch.full((T + 60, 512), 0x7F, dtype=torch.uint8, device="cuda")
    scales = torch.full((T + 60, 8), 255, dtype=torch.uint8, device="cuda")
    big = lb.QuantRows(codes, scales, 264)
    lb.lora_quant_rows(c.x, out=big[30:30 + T])
    assert all(torch.equal(a, b) for a, b in zip(_run(c, big[30:30 + T], lb.lora_backward_quant),
                                                 _run(c, q, lb.lora_backward_quant)))


def test_not_finite_row_stays_with_its_adapter():
    """A NaN in one row's saved input reaches that adapter's dA and nothing else (v is saved)."""
    c = GpuCase(_wl("bf16", [16, 8, 4], 264, 136))
    seg = lb.lora_segments_build(c.ids, 3)
    v = lb.lora_shrink(c.x, c.table, seg)
    q = lb.lora_quant_rows(c.x)
    want = _run(c, q, lb.lora_backward_quant, v)
    row = int(np.nonzero(c.wl.ids == 1)[0][0])
    q.codes[row, 7] = 0x7F
    got = _run(c, q, lb.lora_backward_quant, v)
    assert torch.isnan(got[1][:, 7]).all() and torch.equal(got[1][:, 8:], want[1][:, 8:])
    assert all(torch.equal(a, b) for i, (a, b) in enumerate(zip(got, want)) if i != 1)
