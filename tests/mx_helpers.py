"""The microscaled 4-bit form and the experts' operators in 64 bits on the CPU: the oracle of their tests.  It shares
no code with the library: codes are decoded from their bit fields and encoded by searching the table of the 8
magnitudes, rows move one choice at a time."""
import numpy as np
import torch

import quant_helpers as qh

BLOCK, PAD = 32, 256


def _e2m1_table():
    out = np.empty(16)
    for c in range(16):
        s, e, f = c >> 3, (c >> 1) & 3, c & 1
        mag = (1 + f / 2) * 2.0 ** (e - 1) if e else f / 2
        out[c] = -mag if s else mag
    return out


E2M1 = _e2m1_table()
_POS = E2M1[:8]


def encode_codes(z):
    """Codes of values z with |z| <= 6, nearest, ties to the even code."""
    z = np.asarray(z, np.float64)
    mag = np.abs(z)
    hi = np.clip(np.searchsorted(_POS, mag), 0, 7)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = mag - _POS[lo], _POS[hi] - mag
    c = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    return np.where(np.signbit(z), c + 8, c).astype(np.uint8)


def scale_bytes(top):
    """Exponent bytes of blocks with the largest magnitudes top (255 where that is not finite)."""
    out = np.full(np.shape(top), 127, np.uint8)
    for i, v in np.ndenumerate(top):
        if not np.isfinite(v):
            out[i] = 255
        elif v > 0:
            e = max(-127, int(np.floor(np.log2(v))) - 4)  # (below any answer: 6 * 2^e < v)
            while v > 6 * 2.0 ** e:
                e += 1
            out[i] = e + 127
    return out


def quant(a, square=False):
    """(codes unpacked [n, round_up(k, 256)], scales [n, round_up(k, 256) / 32]) of a, float64 [n, k]."""
    a = np.asarray(a, np.float64)
    n, k = a.shape
    h = BLOCK if square else 1
    p = np.zeros((qh.pad_up(n, h), qh.pad_up(k, PAD)))
    p[:n, :k] = a
    b = p.reshape(p.shape[0] // h, h, p.shape[1] // BLOCK, BLOCK)
    with np.errstate(invalid="ignore"):
        top = np.where(np.isfinite(b).all(axis=(1, 3)), np.abs(b).max(axis=(1, 3)), np.inf)
    s = scale_bytes(top)
    ok = (s != 255)[:, None, :, None]
    with np.errstate(invalid="ignore"):
        z = np.where(ok, np.where(ok, b, 0) / 2.0 ** (s.astype(np.float64) - 127)[:, None, :, None], 0.0)
    codes = encode_codes(z).reshape(p.shape)[:n]
    return codes, np.repeat(s, h, 0)[:n]


def pack(codes):
    return (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)


def unpack(packed):
    packed = np.asarray(packed)
    return np.stack([packed & 15, packed >> 4], -1).reshape(packed.shape[0], -1)


def values(codes, scales, cols):
    """float64 values of unpacked codes and scales (numpy uint8)."""
    with np.errstate(over="ignore"):
        f = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (E2M1[codes] * np.repeat(f, BLOCK, 1)[:, : codes.shape[1]])[:, :cols]


def random_mx(T, d, g, spread=2.0, scale=1.0):
    """(packed codes, scales) of random rows with blocks of different size, as torch tensors on the CPU."""
    x = torch.randn(T, d, generator=g, dtype=torch.float64) * scale
    x *= torch.exp2(torch.randint(-3, 4, (T, 1), generator=g).double() * spread / 3)
    c, s = quant(x.numpy())
    return torch.from_numpy(pack(c)), torch.from_numpy(s)


def random_rows8(T, d, g):
    x = torch.randn(T, d, generator=g, dtype=torch.float64) * torch.exp2(torch.randint(-3, 4, (T, 1), generator=g).double())
    c, s = qh.quant(x.numpy())
    scales = np.full((T, qh.pad_up(s.shape[1], 4)), 127, np.uint8)
    scales[:, : s.shape[1]] = s
    return torch.from_numpy(c), torch.from_numpy(scales)


def product_bound(x, w, y, dtype, bits, wscale=None, xscale=None, y0=None, splits=1):
    """Largest error that y = x w^T in dtype may have, element by element.

    fp32 sums: the products (exact but for 8-bit rows with bf16 y) of a step of 128 columns, the steps and the parts
    of a split k are at most 128 + k / 128 + splits fp32 additions deep, each off by at most 2^-23 of the magnitudes
    added so far (also where the hardware cuts instead of rounding), and the parts of a workgroup's waves 8 more;
    then one addition of y0 and one rounding by half a step.

    8-bit rows with bf16 y: besides, all but the largest of each 8 products are cut at 2^-13 of the power of two at or
    below the largest; wscale, xscale [rows, columns]: the scales, of which a code counts as 1 (weight) and 2^-6 (rows)
    at the least."""
    depth = 128 + -(-x.shape[1] // 128) + splits + 8
    mag = np.abs(x) @ np.abs(w).T
    acc = depth * 2.0 ** -23 * mag + 2.0 ** -126
    if bits == 8 and dtype == torch.bfloat16:
        k8 = qh.pad_up(x.shape[1], 8)
        floor = lambda m, s, least: np.where(m == 0, 0, np.maximum(np.abs(m), least * s))
        top = [np.pad(m, ((0, 0), (0, k8 - m.shape[1]))).reshape(m.shape[0], -1, 8).max(-1)
               for m in (floor(x, xscale, 2.0 ** -6), floor(w, wscale, 1.0))]
        acc = acc + 7 * 2.0 ** -13 * (top[0] @ top[1].T)
    if y0 is not None:
        acc = acc + 2.0 ** -24 * (np.abs(y0) + mag)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    return acc + half * (np.abs(y) + acc)


def expand(scales, block, cols):
    """Scales [rows, blocks] (bytes) as factors [rows, cols]."""
    return np.repeat(2.0 ** (scales.astype(np.float64) - 127), block, 1)[:, :cols]


# ------------------------------------------------------------------ experts


def sort_choices(ids, experts):
    """offsets [E + 1], perm (the choices of an expert, in order), pos [T, k] (-1: none) of ids [T, k]."""
    flat = np.asarray(ids).reshape(-1)
    perm = np.concatenate([np.nonzero(flat == e)[0] for e in range(experts)]) if len(flat) else np.zeros(0, int)
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(experts)])])
    pos = np.full(len(flat), -1)
    pos[perm] = np.arange(len(perm))
    return offsets, perm, pos.reshape(np.shape(ids))


def random_choices(T, k, experts, seed, drop=0.1, skew=1.0):
    """Distinct experts for every token (as far as there are), some chosen more often, some choices dropped."""
    rng = np.random.default_rng(seed)
    like = skew * rng.standard_normal(experts) + rng.gumbel(size=(T, experts))
    order = np.argsort(-like, axis=1)
    ids = np.stack([order[:, j % experts] for j in range(k)], 1) if T else np.zeros((0, k), int)
    return np.where(rng.random(ids.shape) < drop, -1, ids).astype(np.int32)
