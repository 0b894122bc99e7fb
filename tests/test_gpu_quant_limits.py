"""The 8-bit calls at the limits of what their header promises, against 64 bits.

Operands are made of codes and scale bytes directly, so that they hold what
rounded data rarely does."""
import numpy as np
import pytest
import torch

import quant_plans

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expand_token_adapter_amd as lb
    import quant_helpers as qh

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, of the value


def _code(v):
    c = int(qh.encode_codes(np.array([v]))[0])
    assert qh.E4M3[c] == v
    return c


def _operand(codes, byte, weight=False):
    """QuantRows or QuantWeight of codes (numpy uint8 [n, k], k a multiple of 128) with one scale byte."""
    n, k = codes.shape
    scales = torch.full((-(-n // 128) if weight else n, -(-k // 512) * 4), byte, dtype=torch.uint8, device="cuda")
    c = torch.from_numpy(codes).cuda()
    return lb.QuantWeight(c, scales, n, k) if weight else lb.QuantRows(c, scales, k)


def _bound(x, w, want, dt, y0=None, parts=0):
    """Largest error of y (+)= x w^T by the header's rule, for codes with scale byte 127.

    fp32 additions: the 128 products of a block one after another at the worst, then the blocks, the parts of
    a split k and the old value, each addition off by at most 2^-23 of the magnitudes (half of that where it
    rounds); bf16 y: the cut; at last one rounding of y."""
    depth = 128 + x.shape[1] // 128 + parts + 1
    mag = np.abs(x) @ np.abs(w).T + (0 if y0 is None else np.abs(y0))
    acc = depth * 2.0 ** -23 * mag
    if dt == torch.bfloat16:
        X, W = (np.where(m != 0, np.maximum(np.abs(m), 2.0 ** -6), 0).reshape(m.shape[0], -1, 8) for m in (x, w))
        top = np.stack([(X[t] * W).max(-1).sum(-1) for t in range(X.shape[0])])  # [T, N], a group at a time
        acc = acc + 7 * 2.0 ** -13 * top
    return acc + HALF[dt] * (np.abs(want) + acc)


# rows of the streamed weight, and of tiles
@pytest.mark.parametrize("T", [3, 40, 300])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_cancelling_outliers_keep_the_bound(dtype, add, T):
    """Groups of 8 columns in pairs: each has one product of up to 448^2 that the other cancels, beside codes of
    every size (zeros and subnormal codes among them)."""
    dt = TYPES[dtype]
    rng = np.random.default_rng(T)
    N, k = 136, 512
    x, w = (rng.integers(0, 127, size=(m, k)).astype(np.uint8) for m in (T, N))
    for m in (x, w):
        m[:, rng.random(k) < 0.3] &= 15  # subnormal codes and the smallest normal ones
        m[rng.random(m.shape) < 0.5] |= 128
    even = np.arange(0, k, 16)
    at = even + rng.integers(0, 8, size=even.size)
    x[:, at] = rng.integers(100, 127, size=(T, even.size))
    w[:, at] = rng.integers(100, 127, size=(N, even.size))
    x[:, at + 8], w[:, at + 8] = x[:, at], w[:, at] ^ 128
    xv, wv = qh.E4M3[x], qh.E4M3[w]
    y0 = rng.integers(-64, 65, size=(T, N)).astype(np.float64)
    y = torch.from_numpy(y0).to(dt).cuda() if add else None
    got = lb.lora_base_product(_operand(x, 127), _operand(w, 127, True), y=y, accumulate=add, dtype=dt)
    want = xv @ wv.T + (y0 if add else 0)
    off = np.abs(got.double().cpu().numpy() - want)
    assert (off <= _bound(xv, wv, want, dt, y0 if add else None, parts=32)).all()


@pytest.mark.parametrize("T", [1, 64])
@pytest.mark.parametrize("xb,wb", [(1.0, 256.0), (2.0 ** -9, 256.0), (256.0, 2.0 ** -9), (2.0 ** -9, 2.0 ** -6)])
def test_what_is_left_of_small_products(xb, wb, T):
    """One group holds xb * wb and 7 small products, another - xb * wb: their sum is the 7 small ones.  fp32 y has
    them exactly; bf16 y loses no more than the header says."""
    steps = [r for r in range(3, 17) if xb * wb * 2.0 ** -r >= 2.0 ** -18]
    assert steps
    for r in steps:
        small = xb * wb * 2.0 ** -r
        ws = max(small / max(xb * 2.0 ** -(r // 2), 2.0 ** -9), 2.0 ** -9)
        xs = small / ws
        x, w = np.zeros((T, 128), np.uint8), np.zeros((16, 128), np.uint8)
        x[:, 0], x[:, 1:8], x[:, 120] = _code(xb), _code(xs), _code(xb)
        w[:, 0], w[:, 1:8], w[:, 120] = _code(wb), _code(ws), _code(-wb)
        xq, wq = _operand(x, 127), _operand(w, 127, True)
        want = 7 * small
        assert (lb.lora_base_product(xq, wq, dtype=torch.float32) == want).all(), r
        off = (lb.lora_base_product(xq, wq).double() - want).abs().max().item()
        X, W = max(xb, 2.0 ** -6), max(wb, 2.0 ** -6)
        assert off <= 7 * 2.0 ** -13 * X * W * 2 + 2.0 ** -8 * want, r


@pytest.mark.parametrize("T", [16, 127])
@pytest.mark.parametrize("byte,wbyte", [(0, 227), (1, 227), (2, 227), (3, 227), (3, 127), (246, 27), (247, 27), (254, 20)])
def test_products_at_the_ends_of_the_scales(byte, wbyte, T):
    """One code a row times 2^(wbyte - 127): fp32 y takes the value as the bf16 number that a restore gives, bf16 y
    as it is."""
    x, w = np.zeros((T, 128), np.uint8), np.zeros((16, 128), np.uint8)
    x[:, 5] = np.arange(T) if T == 127 else np.arange(T) * 8 + 6
    w[:, 5] = _code(1.0)
    xq, wq = _operand(x, byte), _operand(w, wbyte, True)
    value = torch.from_numpy(qh.E4M3[x[:, 5]] * 2.0 ** (byte - 127))
    times = 2.0 ** (wbyte - 127)
    held = value.float().to(torch.bfloat16)
    assert torch.equal(lb.lora_dequant_rows(xq)[:, 5].cpu(), held)
    got = lb.lora_base_product(xq, wq, dtype=torch.float32).double().cpu()
    assert torch.equal(got, (held.double() * times)[:, None].expand(T, 16))
    assert torch.equal(lb.lora_base_product(xq, wq).double().cpu(), (value * times)[:, None].expand(T, 16))
    assert bool(torch.isinf(held).any()) == (byte >= 247)


@pytest.mark.parametrize("dtype", TYPES)
def test_largest_magnitudes_restore_as_infinity(dtype):
    top = torch.finfo(TYPES[dtype]).max
    x = torch.zeros(3, 128)
    x[0, 0], x[0, 1], x[1, 0], x[2, 0] = top, -top, 1.9375 * 2.0 ** 127, 1.9296875 * 2.0 ** 127
    back = lb.lora_dequant_rows(lb.lora_quant_rows(x.to(TYPES[dtype]).cuda()), torch.float32).cpu()
    assert back[0, 0] == float("inf") and back[0, 1] == -float("inf")
    assert back[1, 0] == float("inf") and back[2, 0] == 1.875 * 2.0 ** 127


# partials of v beside g's: within the room of the partial tiles (two), of the longer set of partials too, and past
# both (two, the last for 8-bit rows too; there lora_backward runs the shrinks in turn unless its buffer is longer)
@pytest.mark.parametrize("dtype,T,d_in,d_out,ranks", [("bf16", 300, 520, 392, (64, 24)), ("f32", 300, 136, 2056, (33, 16)),
                                                      ("f32", 1500, 5128, 136, (128, 9)), ("bf16", 3001, 5128, 5128, (128, 9)),
                                                      ("bf16", 24001, 5128, 5128, (32, 5))])
def test_backward_shrinks_together_and_in_turn(dtype, T, d_in, d_out, ranks):
    """lora_backward in a buffer of its size, in a longer one and with a grant (which always runs the shrinks in
    turn), and lora_backward_quant in a buffer of its size: equal bits, nothing written behind the buffer."""
    dt = TYPES[dtype]
    g = torch.Generator().manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g).to(dt).cuda()
    q = lb.lora_quant_rows(rand(T, d_in))
    x, dy = lb.lora_dequant_rows(q, dt), rand(T, d_out)
    table = lb.AdapterTable([0.05 * rand(r, d_in) for r in ranks], [0.05 * rand(d_out, r) for r in ranks], [2.0, -0.5])
    ids = torch.randint(-1, 2, (T,), generator=g).int().cuda()
    one, status = torch.ones(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(fn, rows, extra, *more):
        query = lb.lora_backward_quant_workspace_bytes if fn is lb.lora_backward_quant else lb.lora_backward_workspace_bytes
        need = query(dt, T, d_in, d_out, max(ranks))
        buf = torch.full((need + extra + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        dA, dB = [torch.ones(r, d_in, device="cuda") for r in ranks], [torch.ones(d_out, r, device="cuda") for r in ranks]
        dx = torch.ones(T, d_in, dtype=dt, device="cuda")
        seg = lb.lora_segments_build(ids, 2)
        fn(rows, dy, table, lb.GradTable(dA, dB), seg, *more, dx=dx, ws=buf[:need + extra])
        torch.cuda.synchronize()
        assert int(seg.err.item()) == 0 and bool((buf[need + extra:] == 0xA5).all())
        return dA + dB + [dx]

    want = run(lb.lora_backward_preemptible, x, 0, one, status)
    assert int(status.item()) == 0
    longer = lb.lora_backward_quant_workspace_bytes(dt, T, d_in, d_out, max(ranks))
    for got in (run(lb.lora_backward, x, 0), run(lb.lora_backward, x, longer)):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    first = run(lb.lora_backward_quant, q, 0)
    assert torch.equal(first[-1], want[-1])  # dX
    assert all(torch.equal(a, b) for a, b in zip(run(lb.lora_backward_quant, q, 1 << 20), first))


# ---------------------------------------------------------------- products through every kernel

def _values(codes, scales, k, rows=1):
    """Values (float64, on the GPU) of codes, and 2^-6 times their blocks' scales."""
    table = torch.from_numpy(qh.E4M3).cuda()
    v = table.index_select(0, codes[:, :k].reshape(-1).int()).view(codes.shape[0], k)
    s = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), scales.int() - 127)
    s = s.repeat_interleave(rows, 0)[: codes.shape[0]].repeat_interleave(128, 1)[:, :k]
    return v * s, s * 2.0 ** -6


def _cut_terms(v, floor):
    """Largest counted magnitude of each group of 8 columns."""
    return torch.where(v != 0, torch.maximum(v.abs(), floor), 0.0).view(v.shape[0], -1, 8).amax(-1)


@pytest.mark.parametrize("dtype,T,k,n,kernel,parts,pieces", quant_plans.PRODUCTS)
def test_product_of_every_kernel(dtype, T, k, n, kernel, parts, pieces):
    """Stored and added, against 64 bits (on the GPU), with ragged edges; nothing beside y changes, and the bits are
    the same a second time."""
    dt = TYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(T + k + n)
    x = torch.randn(T, k, device="cuda", generator=g) * torch.exp(2 * torch.randn(T, 1, device="cuda", generator=g))
    x[:, ::37] *= 30
    xq = lb.lora_quant_rows(x)
    wq = lb.lora_quant_weight(0.02 * torch.randn(n, k, device="cuda", generator=g))
    (xv, xf), (wv, wf) = _values(xq.codes, xq.scales, k), _values(wq.codes, wq.scales, k, 128)
    product, mag = xv @ wv.T, xv.abs() @ wv.abs().T
    cut = 7 * 2.0 ** -13 * (_cut_terms(xv, xf) @ _cut_terms(wv, wf).T) if dtype == "bf16" else 0.0
    y0 = torch.randn(T, n, device="cuda", generator=g).to(dt)
    for add in (False, True):
        y = torch.full((T + 2, n + 8), 3.0, dtype=dt, device="cuda")
        y[1:T + 1, :n] = y0
        lb.lora_base_product(xq, wq, y=y[1:T + 1, :n], accumulate=add)
        want = product + (y0.double() if add else 0.0)
        depth = 128 + -(-k // 128) + parts + 1  # as in _bound
        acc = depth * 2.0 ** -23 * (mag + (y0.double().abs() if add else 0.0)) + cut
        bound = acc + HALF[dt] * (want.abs() + acc)
        off = (y[1:T + 1, :n].double() - want).abs()
        assert bool((off <= bound).all()), (add, float((off / bound).max()))
        assert bool((y[0] == 3).all() and (y[T + 1] == 3).all() and (y[:, n:] == 3).all())
        again = y0.clone()
        lb.lora_base_product(xq, wq, y=again, accumulate=add)
        assert torch.equal(again, y[1:T + 1, :n])
