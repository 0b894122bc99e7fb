"""The 8-bit form and the operators on it, in 64 bits on the CPU: the oracle of the
tests of quantised rows, weights, base product and backward.  It shares no code
with the library: codes are decoded from their bit fields and encoded by
searching the table of the 256 values."""
import numpy as np
import torch

BLOCK = 128


def pad_up(n, m):
    return -(-n // m) * m


def _e4m3_table():
    out = np.empty(256)
    for c in range(256):
        s, e, f = c >> 7, (c >> 3) & 15, c & 7
        mag = (1 + f / 8) * 2.0 ** (e - 7) if e else f / 8 * 2.0 ** -6
        out[c] = np.nan if (e == 15 and f == 7) else (-mag if s else mag)
    return out


E4M3 = _e4m3_table()
_POS = E4M3[:127]  # codes 0 .. 126: ascending magnitudes up to 448


def encode_codes(z):
    """Codes of values z with |z| <= 448 (NaN: 0x7f), nearest, ties to the even code."""
    z = np.asarray(z, np.float64)
    mag = np.where(np.isfinite(z), np.abs(z), 0.0)
    hi = np.clip(np.searchsorted(_POS, mag), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = mag - _POS[lo], _POS[hi] - mag
    c = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.signbit(z), c + 128, c)
    return np.where(np.isfinite(z), c, 127).astype(np.uint8)


def scale_bytes(top):
    """Exponent bytes of blocks with the largest finite magnitudes top."""
    out = np.full(np.shape(top), 127, np.uint8)
    for i, v in np.ndenumerate(top):
        if v > 0:
            e = -127
            while v > 448 * 2.0 ** e:
                e += 1
            out[i] = e + 127
    return out


def _blocks(a, rows):
    """a [n, k] as zero-padded blocks [nb, rows, kb, 128]."""
    n, k = a.shape
    p = np.zeros((pad_up(n, rows), pad_up(k, BLOCK)))
    p[:n, :k] = a
    return p.reshape(p.shape[0] // rows, rows, p.shape[1] // BLOCK, BLOCK)


def quant(a, rows=1):
    """(codes [n, round_up(k, 128)], scales [ceil(n / rows), ceil(k / 128)]) of a, float64 [n, k]."""
    b = _blocks(np.asarray(a, np.float64), rows)
    top = np.where(np.isfinite(b), np.abs(b), 0.0).max(axis=(1, 3))
    s = scale_bytes(top)
    with np.errstate(invalid="ignore"):
        z = b / 2.0 ** (s.astype(np.float64) - 127)[:, None, :, None]
    z = np.where(np.isfinite(b), z, np.nan)
    codes = encode_codes(z).reshape(b.shape[0] * rows, -1)[: a.shape[0]]
    return codes, s


def values(codes, scales, cols, rows=1):
    """float64 values of codes and scales (numpy uint8)."""
    with np.errstate(over="ignore"):
        f = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    f = np.repeat(np.repeat(f, rows, 0)[: codes.shape[0]], BLOCK, 1)[:, : codes.shape[1]]
    return (E4M3[codes] * f)[:, :cols]


def base_bound(x, w, y, dtype, y0=None, splits=1):
    """Largest error that y = x w^T in dtype may have, element by element.

    fp32 y: the products are exact; the 128 of a block, the blocks and the parts
    of a split k are at most 128 + k / 128 + splits fp32 additions deep, each off
    by at most 2^-23 of the magnitudes added so far (also where the hardware cuts
    instead of rounding); then one addition of y0 and one rounding by half a step.

    bf16 y: besides, the matrix instruction cuts all but the largest of each 8
    products at 2^-13 of the power of two at or below the largest; a group's
    largest product is at most the product of the two largest factors.  Groups are
    8 codes that are consecutive in memory."""
    depth = BLOCK + -(-x.shape[1] // BLOCK) + splits
    mag = np.abs(x) @ np.abs(w).T
    acc = depth * 2.0 ** -23 * mag + 2.0 ** -126
    if dtype == torch.bfloat16:
        top = [np.abs(m).reshape(m.shape[0], -1, 8).max(-1) for m in (x, w)]
        acc = acc + 7 * 2.0 ** -13 * (top[0] @ top[1].T)
    if y0 is not None:
        acc = acc + 2.0 ** -24 * (np.abs(y0) + mag)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    return acc + half * (np.abs(y) + acc)
