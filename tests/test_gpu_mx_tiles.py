"""Every kernel of a product with a 4-bit weight (mx_plans pins them on the CPU) with what lies beside its operands:
pitches wider than the rows with NaN behind them, one NaN scale on either side, scale bytes at both ends.  Each against
the ordinary call of the same size, bit for bit.  And workspaces that split products share."""
import pytest
import torch

import mx_helpers as mh
import mx_plans

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expand_token_adapter_amd as lb

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _modes(sizes):
    """(bits, type, cut, ...) of the listed sizes: 8-bit rows with bf16 y take the sizes of fp32 y, whose kernels they
    share, and those listed for bf16 y where they may be cut."""
    out = []
    for s in sizes:
        bits, dtype, rest = s[0], s[1], s[2:]
        out.append((bits, dtype, bits == 8 and dtype == "bf16", *rest))
        if bits == 8 and dtype == "f32":
            out.append((8, "bf16", False, *rest))
    return out


def _random(rows, k, bits, g):
    """Codes of every kind (columns past k zero) and mid-range scales."""
    unit = 256 if bits == 4 else 128
    pad = -(-k // unit) * unit
    if bits == 4:
        c = torch.randint(0, 256, (rows, pad // 2), generator=g, device="cuda").to(torch.uint8)
        c[:, k // 2:] = 0
        s = torch.randint(122, 132, (rows, pad // 32), generator=g, device="cuda").to(torch.uint8)
        s[:, -(-k // 32):] = 127
        return c, s
    c = torch.randint(0, 127, (rows, pad), generator=g, device="cuda") | (torch.randint(0, 2, (rows, pad), generator=g, device="cuda") << 7)
    c[:, k:] = 0
    s = torch.randint(122, 132, (rows, -(-pad // 512) * 4), generator=g, device="cuda")
    return c.to(torch.uint8), s.to(torch.uint8)


def _wide(t, more, fill):
    out = torch.full((t.shape[0], t.shape[1] + more), fill, dtype=torch.uint8, device="cuda")
    out[:, : t.shape[1]] = t
    return out


def _check_all(bits, T, k, n, experts, call, last, g):
    """call(x, w) -> y [T, n], of which the first `last` rows count."""
    xc, xs = _random(T, k, bits, g)
    wc, ws = _random((experts or 1) * n, k, 4, g)
    rows = (lambda c, s: lb.MxRows(c, s, k)) if bits == 4 else (lambda c, s: lb.QuantRows(c, s, k))
    weight = lambda c, s: lb.MxWeight(c, s, n, k, experts=experts)
    want = call(rows(xc, xs), weight(wc, ws))[:last]
    assert bool(torch.isfinite(want).all())
    # pitches wider than the rows
    xw = rows(_wide(xc, 256, 0x77 if bits == 4 else 0x7f), _wide(xs, 8, 255))
    ww = weight(_wide(wc, 384, 0x77), _wide(ws, 24, 255))
    assert torch.equal(call(xw, ww)[:last], want), "pitches"
    # one NaN in the rows, one in the weight
    i, j = int(torch.randint(0, max(last, 1), (1,), generator=g, device="cuda")), int(torch.randint(0, len(wc), (1,), generator=g, device="cuda"))
    b = lambda block: int(torch.randint(0, -(-k // block), (1,), generator=g, device="cuda"))
    xs2, ws2 = xs.clone(), ws.clone()
    xs2[i, b(32 if bits == 4 else 128)] = 255
    got = call(rows(xc, xs2), weight(wc, ws))[:last]
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[i : i + 1] = True
    assert torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], want[~bad]), "NaN row"
    ws2[j, b(32)] = 255
    got = call(rows(xc, xs), weight(wc, ws2))[:last]
    bad = torch.isnan(got)
    assert not bad[:, [c for c in range(n) if c != j % n]].any() and torch.equal(got[~bad], want[~bad]), "NaN weight row"
    if experts is None:
        assert bool(bad[:, j].all())
    # scale bytes at both ends: the codes' own products, whichever side has the large scale
    both = lambda a, c: call(rows(xc, torch.full_like(xs, a)), weight(wc, torch.full_like(ws, c)))[:last]
    want = both(127, 127)
    for a, c in ((254, 0), (0, 254)):
        assert torch.equal(both(a, c), want), (a, c)


@pytest.mark.parametrize("bits,dtype,cut,T,k,n,tile,parts", _modes(mx_plans.PRODUCTS))
def test_products(bits, dtype, cut, T, k, n, tile, parts):
    g = torch.Generator(device="cuda").manual_seed(T + k + n)
    ws = torch.empty(lb.LORA_BASE_PRODUCT_MAX_WORKSPACE, dtype=torch.uint8, device="cuda")

    def call(x, w):
        wide = torch.full((T, n + 8), 7.0, dtype=TYPES[dtype], device="cuda")
        lb.lora_base_product_mx(x, w, y=wide[:, :n], ws=ws, cut=cut)
        assert (wide[:, n:] == 7).all()
        return wide[:, :n]

    _check_all(bits, T, k, n, None, call, T, g)


@pytest.mark.parametrize("bits,dtype,cut,T,E,k,n,tile", _modes(mx_plans.EXPERTS))
def test_experts(bits, dtype, cut, T, E, k, n, tile):
    g = torch.Generator(device="cuda").manual_seed(T + k + n)
    seg = lb.lora_expert_segments(torch.from_numpy(mh.random_choices(T, 1, E, T, drop=0.05 if T > 1 else 0.0)).cuda(), E)
    last = int(seg.offsets[-1])

    def call(x, w):
        wide = torch.full((T, n + 8), 7.0, dtype=TYPES[dtype], device="cuda")
        lb.lora_expert_product_mx(x, w, seg, y=wide[:, :n], cut=cut)
        assert (wide[:, n:] == 7).all() and (wide[last:] == 7).all()
        return wide[:, :n]

    _check_all(bits, T, k, n, E, call, last, g)
    # every row at one expert, the last or the first
    xc, xs = _random(T, k, bits, g)
    wc, ws = _random(E * n, k, 4, g)
    x, w = lb.MxRows(xc, xs, k) if bits == 4 else lb.QuantRows(xc, xs, k), lb.MxWeight(wc, ws, n, k, experts=E)
    xv = (lb.lora_dequant_rows_mx if bits == 4 else lb.lora_dequant_rows)(x, torch.float32).double()  # (exact)
    xf = torch.exp2(xs.double() - 127).repeat_interleave(32 if bits == 4 else 128, 1)[:, :k]
    for e in (E - 1, 0):
        lb.lora_expert_segments(torch.full((T, 1), e, dtype=torch.int32, device="cuda"), E, out=seg)
        rows = slice(e * n, (e + 1) * n)
        wv = lb.lora_dequant_rows_mx(w, torch.float32)[rows].double()
        wf = torch.exp2(ws[rows].double() - 127).repeat_interleave(32, 1)[:, :k]
        want = xv @ wv.t()
        got = lb.lora_expert_product_mx(x, w, seg, dtype=TYPES[dtype], cut=cut)
        assert bool(((got.double() - want).abs() <= _bound(xv, wv, xf, wf, want, TYPES[dtype], cut)).all()), e


def _bound(x, w, xf, wf, want, dt, cut):
    """mx_helpers.product_bound, on the GPU: fp32 sums of at most 128 + k / 128 + 8 steps, each off by 2^-23 of the
    magnitudes added, cut products by 7 * 2^-13 of their group's largest, one rounding."""
    acc = (128 + -(-x.shape[1] // 128) + 9) * 2.0 ** -23 * (x.abs() @ w.abs().t()) + 2.0 ** -126
    if cut:
        top = [torch.where(m == 0, 0.0, torch.maximum(m.abs(), least * f)).view(m.shape[0], m.shape[1] // 8, 8).amax(-1)
               for m, f, least in ((x, xf, 2.0 ** -6), (w, wf, 1.0))]
        acc = acc + 7 * 2.0 ** -13 * (top[0] @ top[1].t())
    return acc + (2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24) * (want.abs() + acc)


SPLIT = {bits: [s[2:5] for s in mx_plans.PRODUCTS if s[:2] == (bits, "f32") and s[6] > 1] for bits in (4, 8)}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bits", [4, 8])
def test_split_products_share_a_workspace(bits, dtype):
    """Captured calls over one workspace, every one with its k in parts, replayed in turn and between eager calls."""
    sizes = SPLIT[bits] if bits == 8 or dtype == "f32" else [s[2:5] for s in mx_plans.PRODUCTS if s[:2] == (4, "bf16") and s[6] > 1]
    assert len(sizes) >= 3
    g = torch.Generator(device="cuda").manual_seed(5)
    ws = torch.empty(lb.LORA_BASE_PRODUCT_MAX_WORKSPACE, dtype=torch.uint8, device="cuda")
    calls = []
    for T, k, n in sizes:
        xc, xs = _random(T, k, bits, g)
        x = lb.MxRows(xc, xs, k) if bits == 4 else lb.QuantRows(xc, xs, k)
        w = lb.MxWeight(*_random(n, k, 4, g), n, k)
        y = torch.zeros(T, n, dtype=TYPES[dtype], device="cuda")
        want = lb.lora_base_product_mx(x, w, dtype=y.dtype).clone()  # (a workspace of its own)
        ws.fill_(0)
        assert torch.equal(lb.lora_base_product_mx(x, w, dtype=y.dtype, ws=ws), want)
        assert bool(ws.any()), "k is in parts"
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lb.lora_base_product_mx(x, w, y=y, ws=ws)
        calls.append((x, w, y, graph, want))
    for _ in range(4):
        for x, w, y, graph, want in calls:
            y.fill_(7)
            graph.replay()
        torch.cuda.synchronize()
        for x, w, y, graph, want in calls:
            assert torch.equal(y, want)
        ws.fill_(255)  # (its contents do not matter)
        for x, w, y, graph, want in calls:
            assert torch.equal(lb.lora_base_product_mx(x, w, dtype=y.dtype, ws=ws), want)
