"""4-bit rows and weights on the GPU against the 64-bit form (mx_helpers): codes, scales and restored values exact,
products within the bound that their sums allow (mx_helpers.product_bound)."""
import numpy as np
import pytest
import torch

import mx_helpers as mh
import quant_helpers as qh

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expand_token_adapter_amd as lb

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rows(T, d, seed, dtype):
    """Rows of different size with a few large columns, a row of zeros and one of tiny values."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, d, generator=g) * torch.exp(2 * torch.randn(T, 1, generator=g))
    x[:, :: 37] *= 30
    if T > 2:
        x[1] = 0
        x[2] *= 1e-40
    return x.to(TYPES[dtype])


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _u8(t):
    return t.cpu().numpy()


def _check(a, q, square=False):
    codes, scales = mh.quant(a, square)
    assert np.array_equal(_u8(q.scales)[:, : scales.shape[1]], scales)
    assert np.array_equal(mh.unpack(_u8(q.codes))[:, : codes.shape[1]], codes)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 8), (1, 256), (3, 136), (17, 264), (70, 1160), (5, 4096), (129, 120), (33, 520)])
def test_rows_codes_scales_and_values(T, d, dtype):
    x = _rows(T, d, 7 * T + d, dtype).cuda()
    q = lb.lora_quant_rows_mx(x)
    _check(_f64(x), q)  # (zeros past d and scales of 1 past the last block among them)
    want = torch.from_numpy(mh.values(mh.unpack(_u8(q.codes)), _u8(q.scales), d))
    for name, dt in TYPES.items():
        got = lb.lora_dequant_rows_mx(q, dt)
        assert got.dtype == dt
        assert torch.equal(got.cpu(), want.to(torch.float32).to(dt)), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_exponent(dtype):
    """Blocks of every magnitude, from fp32's smallest numbers to its largest, on the border between two scales too."""
    g = torch.Generator().manual_seed(3)
    m = torch.rand(277 * 4, 64, generator=g, dtype=torch.float64) * 2 - 1
    e = torch.arange(277).repeat_interleave(4)[:, None].double() - 149
    x = (m * 2.0 ** e).to(TYPES[dtype])
    edge = 1.5 * 2.0 ** e[:, 0]
    x[:, 0] = torch.where(torch.arange(len(x)) % 4 == 0, edge, x[:, 0].double()).to(TYPES[dtype])
    x = x.cuda()
    assert bool(torch.isfinite(x).all())
    _check(_f64(x), lb.lora_quant_rows_mx(x))


def test_every_bf16_pattern():
    """Each finite bf16 value in a block of its neighbours, and each as the second largest of its block."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(2048, 32)
    x = torch.where(torch.isfinite(bits.float()), bits, torch.zeros_like(bits)).cuda()
    _check(_f64(x), lb.lora_quant_rows_mx(x))
    y = x.clone()
    y[:, 0] = (x.float().abs().amax(1) * 3).clamp_max(3e38).to(torch.bfloat16)
    _check(_f64(y), lb.lora_quant_rows_mx(y))


def test_not_finite_values_make_their_block_nan():
    for dtype in TYPES:
        x = _rows(6, 400, 5, dtype)
        x[0, 3], x[0, 200], x[3, 399], x[4] = float("nan"), float("inf"), float("-inf"), float("inf")
        q = lb.lora_quant_rows_mx(x.cuda())
        _check(_f64(x), q)
        bad = torch.zeros(6, 416, dtype=torch.bool)
        bad[:, :400] = ~torch.isfinite(x.float())
        bad = bad.view(6, 13, 32).any(-1).repeat_interleave(32, 1)[:, :400]
        back = lb.lora_dequant_rows_mx(q, torch.float32).cpu()
        assert torch.equal(torch.isnan(back), bad)
        assert not torch.isnan(lb.lora_dequant_rows_mx(q, torch.bfloat16).float().cpu()[~bad]).any()


@pytest.mark.parametrize("byte", [0, 1, 2, 127, 252, 253, 254, 255])
def test_restore_takes_every_scale_byte(byte):
    codes = torch.arange(256, dtype=torch.uint8).view(2, 128).cuda()
    q = lb.MxRows(codes, torch.full((2, 8), byte, dtype=torch.uint8).cuda(), 256)
    want = torch.from_numpy(mh.values(mh.unpack(_u8(codes)), np.full((2, 8), byte, np.uint8), 256))
    for dt in TYPES.values():
        got = lb.lora_dequant_rows_mx(q, dt).cpu()
        ref = want.to(torch.float32).to(dt)
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(got, 7.0), torch.nan_to_num(ref, 7.0))


def test_rows_pitch_slices_and_neighbours():
    x = _rows(40, 264, 11, "bf16").cuda()
    wide = torch.full((40, 320), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :264] = x
    codes = torch.full((40, 384), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((40, 24), 9, dtype=torch.uint8, device="cuda")
    q = lb.MxRows(codes, scales, 264)
    lb.lora_quant_rows_mx(wide[3:20, :264], out=q[3:20])
    whole = lb.lora_quant_rows_mx(x)
    assert torch.equal(codes[3:20, :256], whole.codes[3:20]) and torch.equal(scales[3:20, :16], whole.scales[3:20])
    assert (codes[:3] == 9).all() and (codes[20:] == 9).all() and (codes[:, 256:] == 9).all()
    assert (scales[:3] == 9).all() and (scales[20:] == 9).all() and (scales[:, 16:] == 9).all()
    out = torch.full((40, 320), 5.0, dtype=torch.bfloat16, device="cuda")
    lb.lora_dequant_rows_mx(q[3:20], out=out[3:20, :264])
    assert torch.equal(out[3:20, :264], lb.lora_dequant_rows_mx(whole[3:20]))
    assert (out[:3] == 5).all() and (out[20:] == 5).all() and (out[:, 264:] == 5).all()
    one = lb.lora_quant_rows_mx(x[:1])
    assert torch.equal(lb.lora_dequant_rows_mx(lb.MxRows(codes[3:4, :256], scales[3:4, :16], 264)), lb.lora_dequant_rows_mx(whole[3:4]))
    assert one.codes.shape == (1, 256)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(8, 8), (128, 128), (136, 264), (392, 120), (1032, 520), (40, 72), (256, 256)])
def test_weight_and_its_transpose(n, k, dtype):
    w = (0.02 * _rows(n, k, n + k, dtype).float()).to(TYPES[dtype])
    if n > 100:
        w[70, 40] = float("nan")
    _w = w.cuda()
    q, t = lb.lora_quant_weight_mx(_w), lb.lora_quant_weight_mx(_w, transpose=True)
    _check(_f64(w), q, square=True)
    _check(_f64(w).T, t, square=True)
    assert (t.d_out, t.d_in) == (k, n)
    a, b = lb.lora_dequant_rows_mx(q), lb.lora_dequant_rows_mx(t)
    assert torch.equal(torch.isnan(a), torch.isnan(b.t())) and torch.equal(torch.nan_to_num(a, 3.0), torch.nan_to_num(b.t(), 3.0))


def test_weights_of_experts():
    g = torch.Generator().manual_seed(1)
    w = torch.randn(3, 72, 296, generator=g).to(torch.bfloat16).cuda()
    for tr in (False, True):
        q = lb.lora_quant_weight_mx(w, transpose=tr)
        assert q.experts == 3 and (q.d_out, q.d_in) == ((296, 72) if tr else (72, 296))
        for e in range(3):
            one = lb.lora_quant_weight_mx(w[e], transpose=tr)
            rows = slice(e * q.d_out, (e + 1) * q.d_out)
            assert torch.equal(q.codes[rows], one.codes) and torch.equal(q.scales[rows], one.scales)


def test_the_transpose_in_eight_bits_is_the_same_weight():
    """dX = W^T dY of a weight saved with a scale for each row: its values are 8-bit numbers, transposed too."""
    w = (0.02 * torch.randn(264, 520, generator=torch.Generator().manual_seed(2))).cuda()
    q = lb.lora_quant_rows_mx(w)
    values = lb.lora_dequant_rows_mx(q, torch.float32)
    wt = lb.lora_quant_weight(values, transpose=True)
    back = qh.values(_u8(wt.codes), _u8(wt.scales)[:, :3], 264, 128)
    assert np.array_equal(back, _f64(values).T)


# ------------------------------------------------------------------ products


def _operands(T, k, n, bits, seed):
    """(x, w as the library takes them, their values and scale factors)"""
    g = torch.Generator().manual_seed(seed)
    wc, wsc = mh.random_mx(n, k, g, scale=0.02)
    w = lb.MxWeight(wc.cuda(), wsc.cuda(), n, k)
    wv, wf = mh.values(mh.unpack(wc.numpy()), wsc.numpy(), k), mh.expand(wsc.numpy(), 32, k)
    if bits == 4:
        xc, xsc = mh.random_mx(T, k, g)
        x = lb.MxRows(xc.cuda(), xsc.cuda(), k)
        return x, w, mh.values(mh.unpack(xc.numpy()), xsc.numpy(), k), wv, mh.expand(xsc.numpy(), 32, k), wf
    xc, xsc = mh.random_rows8(T, k, g)
    x = lb.QuantRows(xc.cuda(), xsc.cuda(), k)
    nb = -(-k // 128)
    return x, w, qh.values(xc.numpy(), xsc.numpy()[:, :nb], k), wv, mh.expand(xsc.numpy()[:, :nb], 128, k), wf


# the stream, every tile, split k and odd sizes
SIZES = [(1, 8, 8), (1, 4096, 136), (3, 120, 40), (16, 4096, 264), (16, 264, 1032), (17, 136, 8), (33, 1160, 72), (64, 520, 512),
         (100, 14336, 104), (150, 2056, 776), (257, 4104, 1288), (600, 1928, 1032), (1500, 520, 2056), (2100, 392, 3000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,k,n", SIZES)
def test_product(T, k, n, bits, dtype):
    x, w, xv, wv, xf, wf = _operands(T, k, n, bits, T + k + n)
    dt = TYPES[dtype]
    want = xv @ wv.T
    y = lb.lora_base_product_mx(x, w, dtype=dt)
    off = np.abs(_f64(y) - want)
    assert np.all(off <= mh.product_bound(xv, wv, want, dt, bits, wf, xf, splits=32)), off.max()
    y0 = torch.randn(T, n, generator=torch.Generator().manual_seed(9)).to(dt)
    got = lb.lora_base_product_mx(x, w, y=y0.cuda(), accumulate=True)
    off = np.abs(_f64(got) - want - _f64(y0))
    assert np.all(off <= mh.product_bound(xv, wv, want + _f64(y0), dt, bits, wf, xf, _f64(y0), splits=32)), off.max()
    assert torch.equal(lb.lora_base_product_mx(x, w, dtype=dt), y)


@pytest.mark.parametrize("bits", [4, 8])
def test_rows_are_independent_and_neighbours_are_left(bits):
    T, k, n = 70, 520, 136
    x, w, xv, wv, _, _ = _operands(T, k, n, bits, 4)
    whole = lb.lora_base_product_mx(x, w)
    x.scales[5, 3], w.scales[9, 2] = 255, 255
    y = torch.full((T + 2, n + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    lb.lora_base_product_mx(x, w, y=y[1 : T + 1, :n])
    got = y[1 : T + 1, :n]
    nan = torch.isnan(got)
    want = torch.zeros_like(nan)
    want[5], want[:, 9] = True, True
    assert torch.equal(nan, want) and torch.equal(got[~nan], whole[~nan])
    assert (y[0] == 7).all() and (y[T + 1] == 7).all() and (y[:, n:] == 7).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_product_reads_nothing_past_its_columns(bits):
    """Pitches wider than the rows, with NaN scales and codes behind them."""
    T, k, n = 40, 264, 72
    x, w, _, _, _, _ = _operands(T, k, n, bits, 6)
    want = lb.lora_base_product_mx(x, w)
    wide = lambda t, c, fill: torch.cat([t, torch.full((t.shape[0], c), fill, dtype=torch.uint8, device="cuda")], 1)
    w2 = lb.MxWeight(wide(w.codes, 128, 0x77), wide(w.scales, 8, 255), n, k)
    x2 = lb.MxRows(wide(x.codes, 128, 0x77), wide(x.scales, 8, 255), k) if bits == 4 else \
        lb.QuantRows(wide(x.codes, 128, 0x7f), wide(x.scales, 4, 255), k)
    assert torch.equal(lb.lora_base_product_mx(x2, w2), want)


@pytest.mark.parametrize("T", [3, 70])
def test_fp32_products_of_8_bit_rows_are_exact(T):
    """Products 2^21 apart in one group of eight columns, every code in each place, at the ends of the scales: sums of a
    few terms that fp32 holds exactly come out exact."""
    rng = np.random.default_rng(4)
    k, n = 256, 40
    for xs, ws in ((127, 127), (0, 200), (250, 20)):
        xc = rng.integers(0, 127, size=(T, k)).astype(np.uint8)
        xc |= (rng.integers(0, 2, size=(T, k)) << 7).astype(np.uint8)
        keep = np.zeros((n, k), bool)
        wc = np.zeros((n, k), np.uint8)
        for i in range(n):  # two columns of one group of eight: one addition, of numbers of at most 22 bits together
            c = 8 * rng.integers(0, k // 8) + rng.permutation(8)[:2]
            keep[i, c] = True
            wc[i, c] = rng.integers(1, 16, size=2)
        w = lb.MxWeight(torch.from_numpy(mh.pack(wc)).cuda(), torch.full((n, k // 32), ws, dtype=torch.uint8).cuda(), n, k)
        x = lb.QuantRows(torch.from_numpy(xc).cuda(), torch.full((T, 4), xs, dtype=torch.uint8).cuda(), k)
        want = qh.values(xc, np.full((T, 2), xs, np.uint8), k) @ mh.values(wc, np.full((n, k // 32), ws, np.uint8), k).T
        assert np.array_equal(_f64(lb.lora_base_product_mx(x, w, dtype=torch.float32)), want), (xs, ws)


def test_scales_at_the_ends_of_their_range():
    for bits, dt in ((4, torch.float32), (8, torch.float32), (4, torch.bfloat16), (8, torch.bfloat16)):
        for T in (4, 40):
            x, w, _, _, _, _ = _operands(T, 256, 40, bits, 8)
            x.scales.fill_(0 if bits == 4 else 3)
            w.scales.fill_(247)
            small = lb.lora_base_product_mx(x, w, dtype=dt)
            x.scales.fill_(120 if bits == 4 else 123)
            w.scales.fill_(127)
            assert torch.equal(small, lb.lora_base_product_mx(x, w, dtype=dt)), (bits, dt, T)


def test_the_binding_checks_its_arguments():
    x, w, *_ = _operands(6, 264, 40, 4, 1)
    x8 = lb.lora_quant_rows(torch.zeros(6, 264, device="cuda"))
    with pytest.raises(ValueError):
        lb.lora_base_product_mx(x, lb.lora_quant_rows_mx(torch.zeros(40, 256, device="cuda")).as_weight())
    with pytest.raises(ValueError):
        lb.lora_base_product_mx(x, w, y=torch.zeros(5, 40, device="cuda"))
    with pytest.raises(ValueError):
        lb.lora_base_product_mx(x, w, accumulate=True)
    with pytest.raises(TypeError):
        lb.lora_base_product_mx(x8, lb.lora_quant_weight(torch.zeros(40, 264, device="cuda")))
    with pytest.raises(lb.LoraError):
        lb.lora_base_product_mx(x, w, y=torch.zeros(6, 41, device="cuda")[:, :40])
    with pytest.raises(ValueError):
        lb.lora_quant_rows_mx(torch.zeros(6, 264, device="cuda"), out=x[:3])
    with pytest.raises(TypeError):
        lb.lora_quant_rows_mx(torch.zeros(6, 264, device="cuda", dtype=torch.float16))
    with pytest.raises(TypeError):
        lb.lora_dequant_rows_mx(x8)
    assert lb.lora_base_product_mx(x[:0], w).shape == (0, 40)
