"""8-bit rows and weights on the GPU against the 64-bit form (quant_helpers).

Codes and scales are exact, and so are the restored values (one rounding to
bf16 where a value is no bf16 number).  The base product is held to the bound
that its fp32 sums allow (quant_helpers.base_bound)."""
import numpy as np
import pytest
import torch

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


def _check_rows(x, q):
    T, d = x.shape
    codes, scales = qh.quant(_f64(x))
    assert np.array_equal(_u8(q.scales)[:, : scales.shape[1]], scales)
    assert np.array_equal(_u8(q.codes)[:, : codes.shape[1]], codes)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 8), (1, 128), (3, 136), (17, 264), (70, 1160), (5, 4096), (129, 120)])
def test_rows_codes_scales_and_values(T, d, dtype):
    x = _rows(T, d, 7 * T + d, dtype).cuda()
    q = lb.lora_quant_rows(x)
    _check_rows(x, q)
    want = qh.values(_u8(q.codes), _u8(q.scales)[:, : -(-d // 128)], d)
    for name, dt in TYPES.items():
        got = lb.lora_dequant_rows(q, dt)
        assert got.dtype == dt
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(torch.float32).to(dt)), name
    nb = -(-d // 128)
    assert not _u8(q.codes)[:, d:].any()  # columns past d hold zeros


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_exponent(dtype):
    """Blocks of every magnitude, from fp32's smallest numbers to its largest."""
    g = torch.Generator().manual_seed(3)
    m = torch.rand(277 * 4, 128, generator=g, dtype=torch.float64) * 2 - 1
    e = torch.arange(277).repeat_interleave(4)[:, None].double() - 149
    x = (m * 2.0 ** e).to(TYPES[dtype])
    x[:, 0] = torch.where(torch.arange(len(x)) % 4 == 0, 1.75 * 2.0 ** e[:, 0], x[:, 0].double()).to(TYPES[dtype])  # the step between two scales
    x = x.cuda()
    assert bool(torch.isfinite(x).all())
    _check_rows(x, lb.lora_quant_rows(x))


def test_every_bf16_pattern():
    """Each bf16 value in a block of its neighbours (NaN and infinities among them)."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(512, 128)
    x = bits.cuda()
    q = lb.lora_quant_rows(x)
    codes, scales = qh.quant(_f64(x))
    got = _u8(q.codes).copy()
    nan = np.isnan(qh.E4M3[got])
    assert np.array_equal(nan, ~np.isfinite(_f64(x)))  # what is not finite becomes NaN, and nothing else does
    assert np.array_equal(got[~nan], codes[~nan])
    assert np.array_equal(_u8(q.scales)[:, :1], scales)


def test_not_finite_values_stay_in_their_place():
    x = _rows(6, 400, 5, "f32")
    x[0, 3], x[0, 200], x[3, 5], x[4] = float("nan"), float("inf"), float("-inf"), float("inf")
    q = lb.lora_quant_rows(x.cuda())
    _, scales = qh.quant(_f64(x))
    assert np.array_equal(_u8(q.scales)[:, :4], scales)
    back = lb.lora_dequant_rows(q, torch.float32).cpu()
    assert torch.equal(torch.isnan(back), ~torch.isfinite(x))
    assert (_u8(q.scales)[4, :4] == 127).all()  # a block without a finite value has the scale 1


@pytest.mark.parametrize("byte", [0, 1, 2, 127, 253, 254, 255])
def test_restore_takes_every_scale_byte(byte):
    codes = torch.arange(256, dtype=torch.uint8).view(2, 128).cuda()
    q = lb.QuantRows(codes, torch.full((2, 4), byte, dtype=torch.uint8).cuda(), 128)
    want = torch.from_numpy(qh.values(_u8(codes), np.full((2, 1), byte, np.uint8), 128))
    for dt in TYPES.values():
        got = lb.lora_dequant_rows(q, dt).cpu()
        ref = want.to(torch.float32).to(dt)
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(got, 7.0), torch.nan_to_num(ref, 7.0))


def test_rows_pitch_slices_and_neighbours():
    """A checkpoint filled piece by piece: nothing beside the written rows and columns changes."""
    x = _rows(40, 264, 11, "bf16").cuda()
    wide = torch.full((40, 320), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :264] = x
    codes = torch.full((40, 512), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((40, 8), 9, dtype=torch.uint8, device="cuda")
    q = lb.QuantRows(codes, scales, 264)
    lb.lora_quant_rows(wide[3:20, :264], out=q[3:20])
    whole = lb.lora_quant_rows(x)
    assert torch.equal(codes[3:20, :384], whole.codes[3:20]) and torch.equal(scales[3:20, :3], whole.scales[3:20, :3])
    assert (codes[:3] == 9).all() and (codes[20:] == 9).all() and (codes[:, 384:] == 9).all()
    assert (scales[:3] == 9).all() and (scales[20:] == 9).all() and (scales[:, 3:] == 9).all()
    out = torch.full((40, 320), 5.0, dtype=torch.bfloat16, device="cuda")
    lb.lora_dequant_rows(q[3:20], out=out[3:20, :264])
    assert torch.equal(out[3:20, :264], lb.lora_dequant_rows(whole[3:20]))
    assert (out[:3] == 5).all() and (out[20:] == 5).all() and (out[:, 264:] == 5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(8, 8), (128, 128), (136, 264), (392, 120), (1032, 520)])
def test_weight_and_its_transpose(n, k, dtype):
    w = (0.02 * _rows(n, k, n + k, dtype).float()).to(TYPES[dtype]).cuda()
    codes, scales = qh.quant(_f64(w), 128)
    q = lb.lora_quant_weight(w)
    assert np.array_equal(_u8(q.codes), codes) and np.array_equal(_u8(q.scales)[:, : scales.shape[1]], scales)
    t = lb.lora_quant_weight(w, transpose=True)
    assert (t.d_out, t.d_in) == (k, n)
    assert np.array_equal(_u8(t.codes)[:, :n], codes[:, :k].T) and not _u8(t.codes)[:, n:].any()
    assert np.array_equal(_u8(t.scales)[:, : scales.shape[0]], scales.T)


def _product_case(T, k, n, seed, xs=1.0):
    x = lb.lora_quant_rows((_rows(T, k, seed, "f32") * xs).cuda())
    w = lb.lora_quant_weight((0.02 * torch.randn(n, k, generator=torch.Generator().manual_seed(seed + 1))).cuda())
    xv = qh.values(_u8(x.codes), _u8(x.scales)[:, : -(-k // 128)], k)
    wv = qh.values(_u8(w.codes), _u8(w.scales)[:, : -(-k // 128)], k, 128)
    return x, w, xv, wv


SIZES = [(1, 8, 8), (1, 128, 16), (1, 4096, 264), (2, 136, 72), (15, 520, 136), (16, 1024, 128), (17, 264, 120),
         (33, 640, 392), (64, 1160, 64), (65, 392, 1032), (127, 2048, 136), (130, 256, 520), (257, 776, 264),
         (300, 5128, 128), (5, 16000, 72), (513, 1032, 776), (1029, 264, 1288)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("T,k,n", SIZES)
def test_base_product(T, k, n, add, dtype):
    _check_product(T, k, n, add, dtype)


# every tile and split: about a round of each tile on the chip, with ragged edges along all three sizes
LARGE = [(12, 264, 14344), (40, 10248, 1032), (200, 12000, 264), (520, 520, 4104), (1030, 520, 4104), (2050, 776, 4104),
         (4100, 392, 4104), (300, 33000, 136)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,n", LARGE)
def test_base_product_large(T, k, n, dtype):
    _check_product(T, k, n, T % 4 == 0, dtype)


def _check_product(T, k, n, add, dtype):
    dt = TYPES[dtype]
    x, w, xv, wv = _product_case(T, k, n, T + k + n)
    y0 = torch.randn(T, n, generator=torch.Generator().manual_seed(9)).to(dt)
    y = torch.full((T + 2, n + 8), 3.0, dtype=dt, device="cuda")
    y[1:T + 1, :n] = y0.cuda()
    out = lb.lora_base_product(x, w, y=y[1:T + 1, :n], accumulate=add)
    assert out.data_ptr() == y[1:].data_ptr()
    want = xv @ wv.T + (_f64(y0) if add else 0.0)
    bound = qh.base_bound(xv, wv, want, dt, _f64(y0) if add else None, splits=64)
    off = np.abs(_f64(out) - want)
    assert (off <= bound).all(), f"{(off / bound).max():.3g} of the bound at {np.unravel_index((off / bound).argmax(), off.shape)}"
    assert (y[0] == 3).all() and (y[T + 1] == 3).all() and (y[:, n:] == 3).all()
    again = y0.cuda() if add else None
    again = lb.lora_base_product(x, w, y=again, accumulate=add, dtype=dt)
    assert torch.equal(again, out)  # and the same bits a second time


@pytest.mark.parametrize("T", [1, 40, 300])
def test_base_product_keeps_not_finite_rows_apart(T):
    x, w, xv, wv = _product_case(T, 392, 136, 4)
    want = lb.lora_base_product(x, w, dtype=torch.float32)
    bad = [0, T - 1]
    x.codes[bad[0], 5] = 0x7F
    x.scales[bad[1], 1] = 255
    got = lb.lora_base_product(x, w, dtype=torch.float32)
    assert torch.isnan(got[bad]).all()
    keep = [t for t in range(T) if t not in bad]
    assert torch.equal(got[keep], want[keep])


def test_base_product_of_padded_and_sliced_operands():
    """Operands inside wider buffers whose other bytes are NaN codes."""
    x, w, xv, wv = _product_case(37, 392, 264, 8)
    want = lb.lora_base_product(x, w)
    xc = torch.full((50, 1024), 0x7F, dtype=torch.uint8, device="cuda")
    xs = torch.full((50, 16), 255, dtype=torch.uint8, device="cuda")
    xc[6:43, :512], xs[6:43, :4] = x.codes, x.scales
    wc = torch.full((264, 640), 0x7F, dtype=torch.uint8, device="cuda")
    wsc = torch.full((3, 12), 255, dtype=torch.uint8, device="cuda")
    wc[:, :512], wsc[:, :4] = w.codes, w.scales
    got = lb.lora_base_product(lb.QuantRows(xc, xs, 392)[6:43], lb.QuantWeight(wc, wsc, 264, 392))
    assert torch.equal(got, want)


def test_base_product_of_no_rows():
    x, w, _, _ = _product_case(3, 128, 16, 2)
    assert lb.lora_base_product(x[1:1], w).shape == (0, 16)
    assert lb.lora_dequant_rows(x[2:2]).shape == (0, 128)
    assert len(lb.lora_quant_rows(torch.empty(0, 128, device="cuda"))) == 0


def test_base_product_input_gradient_is_the_transposed_product():
    """dX = W^T dY with the transposed form: the adjoint of the forward product, in 64 bits on the same codes."""
    w = (0.02 * torch.randn(392, 264, generator=torch.Generator().manual_seed(1))).cuda()
    wq, wt = lb.lora_quant_weight(w), lb.lora_quant_weight(w, transpose=True)
    dy = lb.lora_quant_rows(_rows(50, 392, 21, "f32").cuda())
    wv = qh.values(_u8(wq.codes), _u8(wq.scales)[:, :3], 264, 128)
    dv = qh.values(_u8(dy.codes), _u8(dy.scales)[:, :4], 392)
    got = lb.lora_base_product(dy, wt, dtype=torch.float32)
    want = dv @ wv
    assert (np.abs(_f64(got) - want) <= qh.base_bound(dv, wv.T, want, torch.float32)).all()
