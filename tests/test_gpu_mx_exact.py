"""Products of 8-bit rows and a 4-bit weight: exact in both types of y, and cut where the caller allows it.

Every kernel that takes the rows' codes in halves (the listed ones of fp32 y) with outputs whose sums fp32 holds
exactly, so that y is known to the last bit; every kernel that cuts products against the documented bound."""
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
HALVES = [(s[0], *s[2:]) for s in mx_plans.PRODUCTS if s[:2] == (8, "f32")]
HALVES_EXPERTS = [(s[0], *s[2:]) for s in mx_plans.EXPERTS if s[:2] == (8, "f32")]
CUT = [s[2:] for s in mx_plans.PRODUCTS if s[:2] == (8, "bf16")]
CUT_EXPERTS = [s[2:] for s in mx_plans.EXPERTS if s[:2] == (8, "bf16")]


def _rows(T, k, g):
    """Random e4m3 rows, every scale 1, of which column 8 i is the largest number and 8 i + 2 a small one (as large as 2^-5)
    for each i, with the other sign in the odd i: what a group's cut loses."""
    c = torch.randint(0, 127, (T, qh.pad_up(k, 128)), generator=g, device="cuda")
    c |= torch.randint(0, 2, c.shape, generator=g, device="cuda") << 7
    c[:, 0::8] = 126
    c[:, 8::16] |= 128
    c[:, 2::8] = torch.randint(1, 17, c[:, 2::8].shape, generator=g, device="cuda")
    c[:, k:] = 0
    table = torch.from_numpy(np.nan_to_num(qh.E4M3)).cuda()
    scales = torch.full((T, qh.pad_up(c.shape[1] // 128, 4)), 127, dtype=torch.uint8, device="cuda")
    return lb.QuantRows(c.to(torch.uint8), scales, k), table[c][:, :k]


def _weight(n, k, g):
    """Weight rows of four columns, two groups': 6 at the large column of both, which cancel, a code at the small column
    and one at any column of the first.  Every product is a multiple of 2^-10 and their magnitudes add up to less than
    2 * 2688 + 2688 + 1 < 2^13: any order of the sums, in fp32, is exact."""
    pad = qh.pad_up(k, 256)
    c = torch.zeros(n, pad, dtype=torch.uint8, device="cuda")
    pairs = k // 16
    at = 16 * torch.randint(0, max(pairs, 1), (n,), generator=g, device="cuda")
    any_ = at + torch.tensor([1, 3, 4, 5, 6, 7], device="cuda")[torch.randint(0, 6, (n,), generator=g, device="cuda")]
    row = torch.arange(n, device="cuda")
    code = lambda: torch.randint(1, 16, (n,), generator=g, device="cuda").to(torch.uint8)
    c[row, at + 2] = code()
    some = torch.rand(n, generator=g, device="cuda") < 0.5
    c[row[some], any_[some]] = code()[some]
    if pairs:
        c[row, at] = c[row, at + 8] = 7
    scales = torch.full((n, pad // 32), 127, dtype=torch.uint8, device="cuda")
    packed = (c[:, 0::2] | c[:, 1::2] << 4).contiguous()
    return packed, scales, torch.from_numpy(mh.E2M1).cuda()[c.long()][:, :k]


def _old(T, n, dt, g):
    """What is there before: quarters up to 32, so that adding them is exact too (24 bits from 2^-10 to 2^13)."""
    return (torch.randint(-128, 129, (T, n), generator=g, device="cuda") / 4).to(dt)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bits,T,k,n,tile,parts", HALVES)
def test_products_are_exact(bits, T, k, n, tile, parts, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + k + n)
    dt = TYPES[dtype]
    x, xv = _rows(T, k, g)
    wc, ws, wv = _weight(n, k, g)
    w = lb.MxWeight(wc, ws, n, k)
    want = xv @ wv.t()  # (multiples of 2^-10 below 2^13: exact in 64 bits)
    assert torch.equal(lb.lora_base_product_mx(x, w, dtype=dt), want.float().to(dt))
    y0 = _old(T, n, dt, g)
    got = lb.lora_base_product_mx(x, w, y=y0.clone(), accumulate=True)
    assert torch.equal(got, (want + y0.double()).float().to(dt))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bits,T,E,k,n,tile", HALVES_EXPERTS)
def test_experts_products_are_exact(bits, T, E, k, n, tile, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + k + n)
    dt = TYPES[dtype]
    ids = mh.random_choices(T, 1, E, T, drop=0.05, skew=1.0)
    seg = lb.lora_expert_segments(torch.from_numpy(ids).cuda(), E)
    off, perm, _ = mh.sort_choices(ids, E)
    x, xv = _rows(T, k, g)
    wc, ws, wv = _weight(E * n, k, g)
    w = lb.MxWeight(wc, ws, n, k, experts=E)
    y0 = _old(T, n, dt, g)
    for add in (False, True):
        got = lb.lora_expert_product_mx(x, w, seg, y=y0.clone(), accumulate=add)
        for e in range(E):
            a, b = int(off[e]), int(off[e + 1])
            want = xv[a:b] @ wv[e * n : (e + 1) * n].t() + (y0[a:b].double() if add else 0)
            assert torch.equal(got[a:b], want.float().to(dt)), (e, add)
        assert torch.equal(got[len(perm):], y0[len(perm):])


def _bound(xv, wv, want, y0=None, parts=1):
    """mx_helpers.product_bound of 8-bit rows with bf16 y that are cut, every scale 1, on the GPU."""
    depth = 128 + -(-xv.shape[1] // 128) + parts + 8
    mag = xv.abs() @ wv.abs().t()
    acc = depth * 2.0 ** -23 * mag + 2.0 ** -126
    top = [torch.where(m == 0, 0.0, m.abs().clamp_min(least)).view(m.shape[0], m.shape[1] // 8, 8).amax(-1)
           for m, least in ((xv, 2.0 ** -6), (wv, 1.0))]
    acc = acc + 7 * 2.0 ** -13 * (top[0] @ top[1].t())
    if y0 is not None:
        acc = acc + 2.0 ** -24 * (y0.double().abs() + mag)
    return acc + 2.0 ** -8 * (want.abs() + acc)


@pytest.mark.parametrize("T,k,n,tile,parts", CUT)
def test_products_that_may_be_cut_keep_the_bound(T, k, n, tile, parts):
    g = torch.Generator(device="cuda").manual_seed(T + k + n)
    x, xv = _rows(T, k, g)
    wc, ws, wv = _weight(n, k, g)
    w = lb.MxWeight(wc, ws, n, k)
    want = xv @ wv.t()
    got = lb.lora_base_product_mx(x, w, cut=True)
    assert bool(((got.double() - want).abs() <= _bound(xv, wv, want, parts=parts)).all())
    y0 = _old(T, n, torch.bfloat16, g)
    got = lb.lora_base_product_mx(x, w, y=y0.clone(), accumulate=True, cut=True)
    want = want + y0.double()
    assert bool(((got.double() - want).abs() <= _bound(xv, wv, want, y0, parts)).all())


@pytest.mark.parametrize("T,E,k,n,tile", CUT_EXPERTS)
def test_experts_products_that_may_be_cut_keep_the_bound(T, E, k, n, tile):
    g = torch.Generator(device="cuda").manual_seed(T + k + n)
    ids = mh.random_choices(T, 1, E, T, drop=0.05, skew=1.0)
    seg = lb.lora_expert_segments(torch.from_numpy(ids).cuda(), E)
    off, perm, _ = mh.sort_choices(ids, E)
    x, xv = _rows(T, k, g)
    wc, ws, wv = _weight(E * n, k, g)
    y0 = _old(T, n, torch.bfloat16, g)
    got = lb.lora_expert_product_mx(x, lb.MxWeight(wc, ws, n, k, experts=E), seg, y=y0.clone(), cut=True)
    for e in range(E):
        a, b, r = int(off[e]), int(off[e + 1]), slice(e * n, (e + 1) * n)
        want = xv[a:b] @ wv[r].t()
        assert bool(((got[a:b].double() - want).abs() <= _bound(xv[a:b], wv[r], want)).all()), e
    assert torch.equal(got[len(perm):], y0[len(perm):])
