"""Operators of a frozen base in 4 bits and of a mixture of experts, as measurable cases.

A frozen base weight, and the rows that go through it, are held in microscaled
4-bit floating point (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) with
one power-of-two scale per block of 32 along a row:

    value = code * 2^(scale - 127)

A block's scale is the smallest power of two (exponent -127 or more) that brings
its largest magnitude to 6 or less, 1 for a block of zeros; codes are rounded to
nearest, ties to even.  A weight that is used in both directions shares a scale
among 32 x 32 values, so that its transpose holds the same values.  Rows may be
in 8 bits instead (e4m3, one scale per 128 columns).

With a mixture of experts every token chooses k of E experts.  The T k choices
are sorted by expert (stable; a choice of -1 is of no expert), position pos[t, j]
of choice j of token t; rows move there and back with the router's weights.

Operators, each in a plain form (elementary torch operations in 32 bits, rounded
once at the end) and, with ``own`` set, through the library's calls:

    round    rows or a weight -> 4-bit form -> the values that it holds
    product  y (+)= W x from 8-bit or 4-bit rows and a 4-bit weight
    experts  the same with a weight for each expert, rows sorted by expert
    gather   the sort, and y[pos[t, j]] = x[t]; back: dx[t] = sum_j dy[pos[t, j]]
    combine  y[t] = sum_j w[t, j] o[pos[t, j]]; back: do and dw from dy
"""
import math

import torch

own = False

BLOCK = 32
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # layer inputs of a fine-tuning step (4 sequences of 1024 rows, 5120 wide) quantised and read back
        {"name": "round-ft-4096x5120", "op": "round", "rows": 4096, "d": 5120, "dtype": "bf16", "form": "rows"},
        # one short sample's rows of a small fp32 layer, width not a multiple of 32
        {"name": "round-odd-77x1160-f32", "op": "round", "rows": 77, "d": 1160, "dtype": "f32", "form": "rows"},
        # the wide projection's frozen weight, its transpose's form for dX (loading a base model)
        {"name": "round-weight-14336x4096", "op": "round", "rows": 14336, "d": 4096, "dtype": "bf16", "form": "transpose"},
        # one decode row through a square projection: latency and the weight's bytes
        {"name": "product-decode-1x4096", "op": "product", "rows": 1, "d_in": 4096, "d_out": 4096, "bits": 8, "dtype": "bf16", "add": False},
        # an odd number of rows, widths not multiples of a block, fp32 output added to what is there
        {"name": "product-odd-317-add-f32", "op": "product", "rows": 317, "d_in": 5128, "d_out": 1032, "bits": 8, "dtype": "f32", "add": True},
        # the mixed batch (decode rows, prefill segments, fine-tuning rows) through the wide projection, rows in 4 bits
        {"name": "product-mixed-6783", "op": "product", "rows": 6783, "d_in": 4096, "d_out": 14336, "bits": 4, "dtype": "bf16", "add": False},
        # decode of 32 tokens, 4 of 32 narrow experts each: a few rows for every expert, the weights' bytes
        {"name": "experts-decode-32x4of32", "op": "experts", "tokens": 32, "k": 4, "experts": 32, "d_in": 4096, "d_out": 1024,
         "bits": 8, "dtype": "bf16", "drop": False},
        # 2048 fine-tuning tokens, 2 of 8 wide experts each, some choices dropped
        {"name": "experts-ft-2048x2of8", "op": "experts", "tokens": 2048, "k": 2, "experts": 8, "d_in": 4096, "d_out": 14336,
         "bits": 4, "dtype": "bf16", "drop": True},
        # the mixed batch's tokens to 2 of 8 experts
        {"name": "gather-mixed-6783x2of8", "op": "gather", "tokens": 6783, "k": 2, "experts": 8, "d": 4096, "dtype": "bf16", "drop": False, "back": False},
        # the gradient of it for a short ragged fp32 sample, dropped choices
        {"name": "gather-back-odd-211x3-f32", "op": "gather", "tokens": 211, "k": 3, "experts": 12, "d": 1160, "dtype": "f32", "drop": True, "back": True},
        # decode: 8 tokens collect the outputs of 8 experts each
        {"name": "combine-decode-8x8of64", "op": "combine", "tokens": 8, "k": 8, "experts": 64, "d": 4096, "dtype": "bf16", "drop": False, "back": False},
        # the gradient for the fine-tuning rows of a step
        {"name": "combine-back-ft-4096x4of32", "op": "combine", "tokens": 4096, "k": 4, "experts": 32, "d": 4096, "dtype": "bf16", "drop": True, "back": True},
    ]


def _log(rng, lo, hi, step=1):
    hi = max(hi, lo)
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v / step) * step))


def draw(rng):
    op = rng.choice(["round", "product", "product", "experts", "experts", "gather", "combine"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "round":
        return {"op": op, "rows": _log(rng, 1, 1024) * 8 if (form := rng.choice(["rows", "weight", "transpose"])) != "rows" else _log(rng, 1, 8192),
                "d": _log(rng, 8, 5120, 8), "dtype": dtype, "form": form}
    if op == "product":
        return {"op": op, "rows": _log(rng, 1, 6783), "d_in": _log(rng, 256, 14336, 8), "d_out": _log(rng, 256, 4096, 8),
                "bits": rng.choice([4, 8]), "dtype": dtype, "add": rng.random() < 0.5}
    experts = _log(rng, 2, 64)
    c = {"op": op, "tokens": 0, "k": rng.randint(1, min(8, experts)), "experts": experts, "dtype": dtype, "drop": rng.random() < 0.5}
    if op == "experts":
        c["d_in"] = _log(rng, 256, 4096, 8)
        c["d_out"] = _log(rng, 256, min(4096, 200_000_000 // (experts * c["d_in"])), 8)
        return c | {"tokens": _log(rng, 1, 4096 // c["k"]), "bits": rng.choice([4, 8])}
    c["d"] = _log(rng, 8, 8192, 8)
    return c | {"tokens": _log(rng, 1, min(6783, 30_000_000 // (c["k"] * c["d"]))), "back": rng.random() < 0.5}


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    mx = lambda rows, d: rows * (d / 2 + math.ceil(d / BLOCK))
    if op == "round":
        n, d = case["rows"], case["d"]
        form = mx(d, n) if case["form"] == "transpose" else mx(n, d)
        return {"bytes": 2 * (n * d * e + form), "flops": 0}
    if op in ("product", "experts"):
        k, n = case["d_in"], case["d_out"]
        rows = case["rows"] if op == "product" else case["tokens"] * case["k"]
        x = mx(rows, k) if case["bits"] == 4 else rows * (k + math.ceil(k / 128))
        # experts: those that can have rows
        used = 1 if op == "product" else min(case["experts"], rows)
        return {"bytes": x + used * mx(n, k) + rows * n * e * (2 if case.get("add") else 1), "flops": 2 * rows * n * k}
    T, k, d = case["tokens"], case["k"], case["d"]
    if op == "gather":  # (the sort: the choices in, their positions out)
        return {"bytes": (1 + k) * T * d * e + 4 * T * k + (0 if case["back"] else 4 * T * k), "flops": T * k * d if case["back"] else 0}
    if case["back"]:
        return {"bytes": (1 + 2 * k) * T * d * e + 12 * T * k, "flops": 3 * T * k * d}
    return {"bytes": (1 + k) * T * d * e + 8 * T * k, "flops": 2 * T * k * d}


# ---------------------------------------------------------------- the 4-bit form


def _pad(n, m):
    return -(-n // m) * m


def _scale_bytes(amax):
    """Smallest power of two that brings amax to 6 or less, as a byte (exponent + 127); 127 where amax is 0."""
    m, e = torch.frexp(amax)
    byte = (e - 2 - (m <= 0.75).int() + 127).clamp(0, 254)
    return torch.where(amax > 0, byte, torch.full_like(byte, 127))


def _plain_round(x, square=False):
    """The values, in units of their scales, that rows x hold in 4 bits [T, round_up(d, 256)], and the scales' bytes."""
    T, d = x.shape
    tp, dp = _pad(T, BLOCK) if square else T, _pad(d, 256)
    f = torch.zeros(tp, dp, device=x.device, dtype=torch.float32)
    f[:T, :d] = x
    blocks = f.view(tp // BLOCK, BLOCK, -1, BLOCK) if square else f.view(T, 1, -1, BLOCK)
    s = _scale_bytes(blocks.abs().amax((1, 3)))[:, None, :, None]
    z = torch.ldexp(blocks, 127 - s)
    a = z.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    units = (torch.round(z / step) * step).view(tp, dp)[:T]
    return units, s.to(torch.uint8).expand(-1, blocks.shape[1], -1, -1).reshape(tp, dp // BLOCK)[:T]


def _pack(units):
    """Two codes a byte, the lower column in the low four bits."""
    a = units.abs()
    code = torch.where(a <= 2, 2 * a, torch.where(a <= 4, a + 2, torch.full_like(a, 7.0))).to(torch.uint8)
    code |= torch.signbit(units).to(torch.uint8) << 3
    return (code[:, 0::2] | code[:, 1::2] << 4).contiguous()


def _plain_values(codes, scales, d):
    """The 32-bit values that codes and scales stand for."""
    both = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1).int()
    mag = both & 7
    a = torch.where(mag <= 4, 0.5 * mag.float(), torch.where(mag == 7, 6.0, mag.float() - 2))
    f = torch.where(both > 7, -a, a).view(codes.shape[0], -1, BLOCK)
    return torch.ldexp(f, scales[:, :, None].int() - 127).view(codes.shape[0], -1)[:, :d]


def _plain_rows8(codes, scales, d):
    """The 32-bit rows that e4m3 codes and a scale per 128 columns stand for."""
    f = codes.view(torch.float8_e4m3fn).float().view(codes.shape[0], -1, 128)
    return torch.ldexp(f, scales[:, : f.shape[1], None].int() - 127).view(codes.shape[0], -1)[:, :d]


# ---------------------------------------------------------------- inputs


def _activations(T, d, g, dev):
    """Rows as a layer's input has them: rows of different size, a few channels far larger than the rest."""
    x = torch.randn(T, d, generator=g, device=dev)
    x *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device=dev))
    x *= torch.where(torch.rand(1, d, generator=g, device=dev) < 0.004, 20.0, 1.0)
    return x


def _rows8(x):
    """e4m3 codes [T, round_up(d, 128)] and scale bytes [T, round_up(d / 128, 4)] of rows x."""
    T, d = x.shape
    nb = -(-d // 128)
    blocks = torch.zeros(T, nb * 128, device=x.device)
    blocks[:, :d] = x
    blocks = blocks.view(T, nb, 128)
    m, e = torch.frexp(blocks.abs().amax(-1))
    byte = (e - 8 - (m <= 0.875).int() + 127).clamp(0, 254)
    byte = torch.where(m > 0, byte, torch.full_like(byte, 127))
    scales = torch.full((T, _pad(nb, 4)), 127, device=x.device, dtype=torch.uint8)
    scales[:, :nb] = byte.to(torch.uint8)
    return torch.ldexp(blocks, 127 - byte[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(T, -1), scales


def _choices(case, g, dev):
    """Experts of every token [T, k]: distinct, some experts chosen far more often; -1: dropped."""
    E, T = case["experts"], case["tokens"]
    liking = torch.randn(E, generator=g, device=dev) + torch.randn(T, E, generator=g, device=dev)
    ids = liking.topk(case["k"], dim=1).indices.int()
    if case["drop"]:
        ids = torch.where(torch.rand(ids.shape, generator=g, device=dev) < 0.1, -1, ids)
    return ids


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt, op = TYPES[case["dtype"]], case["op"]
    s = {"case": case, "dtype": dt}
    if op == "round":
        s["x"] = (_activations(case["rows"], case["d"], g, dev) if case["form"] == "rows" else
                  0.02 * torch.randn(case["rows"], case["d"], generator=g, device=dev)).to(dt)
        return s
    if op != "product":
        s["ids"] = _choices(case, g, dev)
        s["rows"] = case["tokens"] * case["k"]
    if op in ("product", "experts"):
        k, n, E = case["d_in"], case["d_out"], case.get("experts", 1)
        x = _activations(case["rows"] if op == "product" else s["rows"], k, g, dev)
        if case["bits"] == 4:
            units, s["scales"] = _plain_round(x)
            s["codes"] = _pack(units)
        else:
            s["codes"], s["scales"] = _rows8(x)
        parts = [_plain_round(0.02 * torch.randn(n, k, generator=g, device=dev)) for _ in range(E)]
        s["wcodes"] = torch.cat([_pack(p[0]) for p in parts])
        s["wscales"] = torch.cat([p[1] for p in parts])
        s["y"] = torch.randn(case["rows"], n, generator=g, device=dev).to(dt) if case.get("add") else None
        return s
    T, d, back = case["tokens"], case["d"], case["back"]
    if op == "gather" and not back:
        s["x"] = _activations(T, d, g, dev).to(dt)
    elif op == "gather":
        s["dy"] = torch.randn(s["rows"], d, generator=g, device=dev).to(dt)
    else:
        s["w"] = torch.softmax(torch.randn(T, case["k"], generator=g, device=dev), 1)
        s["o"] = torch.randn(s["rows"], d, generator=g, device=dev).to(dt)
        s["dy"] = torch.randn(T, d, generator=g, device=dev).to(dt) if back else None
    return s


def _plain_sort(ids, experts):
    """offsets [E + 1], the choices in sorted order, and their positions [T, k] (-1: of no expert)."""
    key = torch.where(ids < 0, experts, ids).view(-1)
    order = torch.argsort(key, stable=True)
    offsets = (key[None, :] < torch.arange(experts + 1, device=ids.device)[:, None]).sum(1)
    at = torch.empty_like(order)
    at[order] = torch.arange(order.numel(), device=ids.device)
    return offsets.int(), order, torch.where(ids < 0, -1, at.view(ids.shape)).int()


def prepare(case, seed):
    s = _inputs(case, seed)
    dev, op, dt = torch.device("cuda"), case["op"], s["dtype"]
    if op == "round":
        n, d = case["rows"], case["d"]
        rows, cols = (d, n) if case["form"] == "transpose" else (n, d)
        s["codes"] = torch.zeros(rows, _pad(cols, 256) // 2, device=dev, dtype=torch.uint8)
        s["scales"] = torch.full((rows, _pad(cols, 256) // BLOCK), 127, device=dev, dtype=torch.uint8)
        s["out"] = torch.empty(rows, cols, device=dev, dtype=dt)
    elif op == "product":
        s["out"] = torch.empty(case["rows"], case["d_out"], device=dev, dtype=dt)
    else:
        # rows of no expert lie behind the last expert's and are left as they are
        if op == "experts":
            s["out"] = torch.zeros(s["rows"], case["d_out"], device=dev, dtype=dt)
        elif op == "gather":
            s["out"] = torch.zeros(case["tokens"] if case["back"] else s["rows"], case["d"], device=dev, dtype=dt)
        else:
            s["out"] = torch.zeros(s["rows"] if case["back"] else case["tokens"], case["d"], device=dev, dtype=dt)
            s["dw"] = torch.empty(case["tokens"], case["k"], device=dev)
        s["offsets"], s["order"], s["pos"] = _plain_sort(s["ids"], case["experts"])
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    if own:
        # what a program keeps: the views of the rows and weights, the workspace, and, behind the
        # first call of a layer, the choices' grouping by expert
        import expand_token_adapter_amd as lb

        if op == "round":
            s["mx"] = (lb.MxRows(s["codes"], s["scales"], s["out"].shape[1]) if case["form"] == "rows" else
                       lb.MxWeight(s["codes"], s["scales"], *s["out"].shape))
        elif op in ("product", "experts"):
            k, n, E = case["d_in"], case["d_out"], case.get("experts")
            s["x"] = (lb.MxRows if case["bits"] == 4 else lb.QuantRows)(s["codes"], s["scales"], k)
            s["weight"] = lb.MxWeight(s["wcodes"], s["wscales"], n, k, experts=E)
            if op == "product":
                s["ws"] = torch.empty(lb.lora_base_product_mx_workspace_bytes(case["rows"], k, n), device=dev, dtype=torch.uint8)
        if op in ("experts", "gather", "combine"):
            s["seg"] = lb.lora_expert_segments(s["ids"], case["experts"])
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import expand_token_adapter_amd as lb

        if op == "round":
            if case["form"] == "rows":
                lb.lora_quant_rows_mx(s["x"], out=s["mx"])
            else:
                lb.lora_quant_weight_mx(s["x"], transpose=case["form"] == "transpose", out=s["mx"])
            return {"values": lb.lora_dequant_rows_mx(s["mx"], out=s["out"]), "scales": s["scales"]}
        if op == "product":
            if s["y"] is not None:
                s["out"].copy_(s["y"])  # the call adds to what is there
            return lb.lora_base_product_mx(s["x"], s["weight"], y=s["out"], accumulate=s["y"] is not None, ws=s["ws"])
        if op == "experts":
            return lb.lora_expert_product_mx(s["x"], s["weight"], s["seg"], y=s["out"])
        if op == "gather":
            if case["back"]:
                return lb.lora_expert_gather_backward(s["dy"], s["seg"], dx=s["out"])
            seg = lb.lora_expert_segments(s["ids"], case["experts"], out=s["seg"])
            return {"y": lb.lora_expert_gather(s["x"], seg, y=s["out"]), "offsets": seg.offsets, "pos": seg.pos}
        if case["back"]:
            d_o, dw = lb.lora_expert_combine_backward(s["dy"], s["o"], s["w"], s["seg"], d_o=s["out"], dw=s["dw"])
            return {"do": d_o, "dw": dw}
        return lb.lora_expert_combine(s["o"], s["w"], s["seg"], y=s["out"])

    dt = s["dtype"]
    if op == "round":
        x = s["x"].t() if case["form"] == "transpose" else s["x"]
        units, scales = _plain_round(x, square=case["form"] != "rows")
        blocks = units.view(units.shape[0], -1, BLOCK)
        values = torch.ldexp(blocks, scales[:, :, None].int() - 127).view(units.shape)
        return {"values": values[:, : x.shape[1]].to(dt), "scales": scales}
    if op in ("product", "experts"):
        k, n = case["d_in"], case["d_out"]
        x = (_plain_values if case["bits"] == 4 else _plain_rows8)(s["codes"], s["scales"], k)
        w = _plain_values(s["wcodes"], s["wscales"], k)
        if op == "product":
            y = x @ w.t()
            return (y if s["y"] is None else s["y"].float() + y).to(dt)
        # every expert's rows side by side, padded to the longest group's
        at = s["offsets"][:-1, None].long() + torch.arange(s["most"], device=x.device)
        fits = at < s["offsets"][1:, None]
        y = torch.bmm(x[at.clamp_max(len(x) - 1)], w.view(case["experts"], n, k).transpose(1, 2))
        out = torch.zeros(len(x) + 1, n, device=x.device)
        out[torch.where(fits, at, len(x))] = y
        return torch.where((torch.arange(len(x), device=x.device) < s["offsets"][-1])[:, None], out[:-1], s["out"].float()).to(dt)
    if op == "gather" and not case["back"]:
        offsets, order, pos = _plain_sort(s["ids"], case["experts"])
        on = torch.arange(s["rows"], device=order.device) < offsets[-1]
        return {"y": torch.where(on[:, None], s["x"][order // case["k"]], s["out"]), "offsets": offsets, "pos": pos}
    there = (s["pos"] >= 0)[..., None]
    pos = s["pos"].clamp_min(0).long()
    if op == "gather":
        return torch.where(there, s["dy"][pos].float(), 0.0).sum(1).to(dt)
    rows = torch.where(there, s["o"][pos].float(), 0.0)
    if not case["back"]:
        return (s["w"][..., None] * rows).sum(1).to(dt)
    dy = s["dy"].float()
    on = torch.arange(s["rows"], device=dy.device) < s["offsets"][-1]
    d_o = (s["w"].view(-1, 1) * dy.repeat_interleave(case["k"], 0))[s["order"]]
    return {"do": torch.where(on[:, None], d_o.to(dt), s["out"]), "dw": (rows * dy[:, None]).sum(2)}


# ---------------------------------------------------------------- the definition, in 64 bits


_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_units(z):
    """The nearest of the magnitudes, the one with the even number where two are as near, with z's sign."""
    table = torch.tensor(_MAGNITUDES, device=z.device, dtype=torch.float64)
    a = z.abs().contiguous()
    hi = torch.searchsorted(table, a).clamp(0, 7)
    lo = (hi - 1).clamp_min(0)
    below, above = a - table[lo], table[hi] - a
    take = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return torch.copysign(table[take], z)


def _exact_round(x, square):
    T, d = x.shape
    tp, dp = _pad(T, BLOCK), _pad(d, 256)
    f = torch.nn.functional.pad(x.double(), (0, dp - d, 0, tp - T))
    h = BLOCK if square else 1
    top = f.abs().view(tp // h, h, dp // BLOCK, BLOCK).amax((1, 3))
    e = torch.ceil(torch.log2(top.clamp_min(1e-300) / 6)).clamp(-127, 127)
    e = torch.where(top > 6 * torch.exp2(e), e + 1, e)  # (log2's own rounding)
    e = torch.where((top <= 6 * torch.exp2(e - 1)) & (e > -127), e - 1, e)
    e = torch.where(top > 0, e, torch.zeros_like(e)).repeat_interleave(h, 0)
    scale = torch.exp2(e).repeat_interleave(BLOCK, 1)
    return (_exact_units(f / scale) * scale)[:T, :d], (e + 127).to(torch.uint8)[:T]


def _exact_values(codes, scales, d):
    """e2m1 codes bit by bit: sign, 2 exponent bits (bias 1), 1 bit of fraction."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(1).int()
    e, f = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e > 0, torch.exp2(e.double() - 1) * (1 + f / 2), f / 2)
    return (torch.where(c > 7, -mag, mag) * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, 1))[:, :d]


def _exact_rows8(codes, scales, d):
    """e4m3 codes bit by bit: sign, 4 exponent bits (bias 7), 3 bits of fraction."""
    c = codes.int()
    e, f = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, torch.exp2(e.double() - 7) * (1 + f / 8), f / 512)
    scale = torch.exp2(scales.double() - 127).repeat_interleave(128, 1)[:, : c.shape[1]]
    return (torch.where(c > 127, -mag, mag) * scale)[:, :d]


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "round":
        x = s["x"].t() if case["form"] == "transpose" else s["x"]
        values, scales = _exact_round(x, case["form"] != "rows")
        return {"values": values, "scales": scales}
    if op in ("product", "experts"):
        k, n = case["d_in"], case["d_out"]
        x = (_exact_values if case["bits"] == 4 else _exact_rows8)(s["codes"], s["scales"], k)
        if op == "product":
            y = x @ _exact_values(s["wcodes"], s["wscales"], k).t()
            return y if s["y"] is None else y + s["y"].double()
    E, k = case.get("experts"), case.get("k")
    key = s["ids"].view(-1).long()
    at = [torch.nonzero(key == e)[:, 0] for e in range(E)]  # choices of each expert, in order
    order = torch.cat(at)
    if op == "experts":
        y = torch.zeros(s["rows"], case["d_out"], device=x.device, dtype=torch.float64)
        first = 0
        for e, a in enumerate(at):
            w = _exact_values(*(s[v].view(E, case["d_out"], -1)[e] for v in ("wcodes", "wscales")), case["d_in"])
            y[first : first + len(a)] = x[first : first + len(a)] @ w.t()
            first += len(a)
        return y
    T, d = case["tokens"], case["d"]
    if op == "gather" and not case["back"]:
        y = torch.zeros(s["rows"], d, device=key.device, dtype=torch.float64)
        y[: len(order)] = s["x"].double()[order // k]
        pos = torch.full_like(key, -1)
        pos[order] = torch.arange(len(order), device=key.device)
        offsets = torch.tensor([0] + [len(a) for a in at], device=key.device).cumsum(0)
        return {"y": y, "offsets": offsets.int(), "pos": pos.view(T, k).int()}
    rows = torch.zeros(T * k, d, device=key.device, dtype=torch.float64)
    rows[order] = s["dy" if op == "gather" else "o"].double()[: len(order)]
    rows = rows.view(T, k, d)
    if op == "gather":
        return rows.sum(1)
    w = s["w"].double()
    if not case["back"]:
        return torch.matmul(w[:, None], rows)[:, 0]
    dy = s["dy"].double()
    d_o = torch.zeros(T * k, d, device=key.device, dtype=torch.float64)
    d_o[: len(order)] = (w[..., None] * dy[:, None]).view(T * k, d)[order]
    return {"do": d_o, "dw": torch.matmul(rows, dy[..., None])[..., 0]}
