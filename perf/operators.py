"""The 8-bit operators beside the adapter path, as measurable cases.

A frozen base weight and the fine-tuning rows' saved layer inputs are held in
8-bit floating point (e4m3) with one power-of-two scale per block of 128:

    value = code * 2^(scale - 127)

rows (activations) have one scale per row and 128 columns, weights one per 128
x 128 block.  A block's scale is the smallest power of two (exponent -127 or
more) that brings its largest finite magnitude to 448 or less, and 1 where
there is none; codes are rounded to nearest, ties to even.

Four operators, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and, with ``own`` set, through the library's calls:

    save      rows -> codes and scales (the activation checkpoint)
    restore   codes and scales -> rows
    base      y (+)= x W^T from 8-bit rows and an 8-bit weight
    backward  dA, dB and dX of the adapters from 8-bit saved rows and dY
"""
import math

import torch

own = False

BLOCK = 128
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # saving the layer input of a fine-tuning step: 4 sequences of 1024 rows, 5120 wide
        {"name": "save-ft-4096x5120", "op": "save", "rows": 4096, "d": 5120, "dtype": "bf16"},
        # one short sample's rows of a small fp32 layer, width not a multiple of 128
        {"name": "save-odd-77x1160-f32", "op": "save", "rows": 77, "d": 1160, "dtype": "f32"},
        # the saved inputs of the mixed batch's fine-tuning rows, restored for the layer's recompute
        {"name": "restore-ft-2048x4096", "op": "restore", "rows": 2048, "d": 4096, "dtype": "bf16"},
        # a short ragged sample restored to fp32
        {"name": "restore-odd-333x1416-f32", "op": "restore", "rows": 333, "d": 1416, "dtype": "f32"},
        # one decode row through a square projection: latency and the weight's bytes
        {"name": "base-decode-1x4096", "op": "base", "rows": 1, "d_in": 4096, "d_out": 4096, "dtype": "bf16", "add": False},
        # the decode batch of 256 rows through the same projection
        {"name": "base-decode-256x4096", "op": "base", "rows": 256, "d_in": 4096, "d_out": 4096, "dtype": "bf16", "add": False},
        # an odd number of rows, widths not multiples of 128, fp32 output added to what is there
        {"name": "base-odd-317-add-f32", "op": "base", "rows": 317, "d_in": 5128, "d_out": 1032, "dtype": "f32", "add": True},
        # the mixed batch (decode rows, prefill segments, fine-tuning rows) through the wide projection
        {"name": "base-mixed-6783", "op": "base", "rows": 6783, "d_in": 4096, "d_out": 14336, "dtype": "bf16", "add": False},
        # its backward: dX += dY W of the 2048 fine-tuning rows (the transposed weight, contraction over 14336)
        {"name": "base-dx-2048-add", "op": "base", "rows": 2048, "d_in": 14336, "d_out": 4096, "dtype": "bf16", "add": True},
        # the fine-tuning step's adapter backward: one rank-16 adapter, v kept from the forward
        {"name": "backward-ft-4096x5120", "op": "backward", "rows": 4096, "d_in": 5120, "d_out": 5120, "dtype": "bf16",
         "ranks": "16", "save_v": True, "dx": True},
        # fine-tuning rows of four adapters of different ranks on the wide projection, v recomputed from the 8-bit rows
        {"name": "backward-mixed-2048", "op": "backward", "rows": 2048, "d_in": 4096, "d_out": 14336, "dtype": "bf16",
         "ranks": "8,16,32,64", "save_v": False, "dx": True},
        # a short ragged fp32 batch, odd ranks, first layer (no dX)
        {"name": "backward-odd-211-f32", "op": "backward", "rows": 211, "d_in": 1160, "d_out": 776, "dtype": "f32",
         "ranks": "5,12", "save_v": False, "dx": False},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v / step) * step))


def draw(rng):
    op = rng.choice(["save", "restore", "base", "base", "backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("save", "restore"):
        return {"op": op, "rows": _log(rng, 1, 8192), "d": _log(rng, 8, 14336, 8), "dtype": dtype}
    if op == "base":
        return {"op": op, "rows": _log(rng, 1, 6783), "d_in": _log(rng, 256, 14336, 8), "d_out": _log(rng, 256, 4096, 8),
                "dtype": dtype, "add": rng.random() < 0.5}
    ranks = ",".join(str(rng.choice([4, 8, 13, 16, 32, 64])) for _ in range(rng.randint(1, 6)))
    return {"op": op, "rows": _log(rng, 1, 4096), "d_in": _log(rng, 256, 5120, 8), "d_out": _log(rng, 256, 14336, 8),
            "dtype": dtype, "ranks": ranks, "save_v": rng.random() < 0.5, "dx": rng.random() < 0.8}


def work(case):
    T, e = case["rows"], 2 if case["dtype"] == "bf16" else 4
    q8 = lambda rows, d: rows * (d + math.ceil(d / BLOCK))
    if case["op"] in ("save", "restore"):
        return {"bytes": T * case["d"] * e + q8(T, case["d"]), "flops": 0}
    k, n = case["d_in"], case["d_out"]
    if case["op"] == "base":
        weight = n * k + math.ceil(n / BLOCK) * math.ceil(k / BLOCK)
        return {"bytes": q8(T, k) + weight + T * n * e * (2 if case["add"] else 1), "flops": 2 * T * n * k}
    r = [int(v) for v in case["ranks"].split(",")]
    R, rm = sum(r), sum(r) / len(r)  # each row meets one adapter: the mean rank
    byte = q8(T, k) + T * n * e + R * (k + n) * (e + 4) + (T * k * e if case["dx"] else 0) + (4 * T * rm if case["save_v"] else 0)
    # g and dB read dY, dA the rows; v recomputed reads them again, dX writes its rows
    return {"bytes": byte, "flops": 2 * T * rm * (2 * n + k + (0 if case["save_v"] else k) + (k if case["dx"] else 0))}


# ---------------------------------------------------------------- the 8-bit form


def _pad(n, m):
    return -(-n // m) * m


def _codes(x, scale):
    """Codes (e4m3) of x with one exponent byte per element of `scale`, which broadcasts against x."""
    return torch.ldexp(x, 127 - scale.int()).to(torch.float8_e4m3fn)


def _scale_bytes(amax):
    """Smallest power of two that brings amax to 448 or less, as a byte (exponent + 127); 127 where amax is 0."""
    m, e = torch.frexp(amax)
    byte = (e - 8 - (m <= 0.875).int() + 127).clamp(0, 254)
    return torch.where(amax > 0, byte, torch.full_like(byte, 127)).to(torch.uint8)


def _plain_save(x):
    """Codes [T, round_up(d, 128)] as e4m3 and scales [T, round_up(d / 128, 4)] of rows x."""
    T, d = x.shape
    ld, nb = _pad(d, BLOCK), -(-d // BLOCK)
    f = torch.zeros(T, ld, device=x.device, dtype=torch.float32)
    f[:, :d] = x
    blocks = f.view(T, nb, BLOCK)
    s = _scale_bytes(torch.where(torch.isfinite(blocks), blocks.abs(), torch.zeros_like(blocks)).amax(-1))
    scales = torch.full((T, _pad(nb, 4)), 127, device=x.device, dtype=torch.uint8)
    scales[:, :nb] = s
    return _codes(blocks, s[:, :, None]).view(T, ld), scales


def _plain_rows(codes, scales, d):
    """The 32-bit rows that codes and scales stand for."""
    T, ld = codes.shape
    f = codes.view(torch.float8_e4m3fn).float().view(T, ld // BLOCK, BLOCK)
    return torch.ldexp(f, scales[:, : ld // BLOCK, None].int() - 127).view(T, ld)[:, :d]


def _plain_weight(codes, scales, n, k):
    """The 32-bit weight that codes and 128 x 128 block scales stand for."""
    ld = codes.shape[1]
    s = scales[:, : ld // BLOCK].int().repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1) - 127
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), s)[:, :k]


# ---------------------------------------------------------------- inputs


def _activations(T, d, g, dev):
    """Rows as a layer's input has them: rows of different size, a few channels far larger than the rest."""
    x = torch.randn(T, d, generator=g, device=dev)
    x *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device=dev))
    x *= torch.where(torch.rand(1, d, generator=g, device=dev) < 0.004, 20.0, 1.0)
    return x


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    T, dt = case["rows"], TYPES[case["dtype"]]
    s = {"case": case, "dtype": dt}
    if case["op"] == "save":
        s["x"] = _activations(T, case["d"], g, dev).to(dt)
        return s
    d = case["d"] if case["op"] == "restore" else case["d_in"]
    x = _activations(T, d, g, dev)
    if case["op"] == "base" and case["add"]:
        x *= 0.01  # gradients of the layer's output
    codes, scales = _plain_save(x)
    s["codes"], s["scales"] = codes.view(torch.uint8), scales
    if case["op"] == "restore":
        return s
    n = case["d_out"]
    if case["op"] == "base":
        w = torch.zeros(_pad(n, BLOCK), _pad(d, BLOCK), device=dev)
        w[:n, :d] = 0.02 * torch.randn(n, d, generator=g, device=dev)
        nb, kb = w.shape[0] // BLOCK, w.shape[1] // BLOCK
        blocks = w.view(nb, BLOCK, kb, BLOCK)
        b = _scale_bytes(blocks.abs().amax((1, 3)))
        s["wcodes"] = _codes(blocks, b[:, None, :, None]).view(torch.uint8).view(w.shape)[:n].contiguous()
        s["wscales"] = torch.full((nb, _pad(kb, 4)), 127, device=dev, dtype=torch.uint8)
        s["wscales"][:, :kb] = b
        s["y"] = torch.randn(T, n, generator=g, device=dev).to(dt) if case["add"] else None
        return s
    ranks = [int(r) for r in case["ranks"].split(",")]
    # samples of consecutive rows, one adapter each; in batches of several adapters some rows have none
    A, samples = len(ranks), min(T, 2 * len(ranks))
    sample = torch.arange(T, device=dev) * samples // T
    who = torch.randint(0, A + 1 if A > 2 else A, (samples,), generator=g, device=dev)
    s["ids"] = torch.where(who < A, who, -1)[sample].int()
    s["ranks"], s["rates"] = ranks, [32.0 / r for r in ranks]  # alpha / rank
    s["A"] = [(0.02 * torch.randn(r, d, generator=g, device=dev)).to(dt) for r in ranks]
    s["B"] = [(0.02 * torch.randn(n, r, generator=g, device=dev)).to(dt) for r in ranks]
    s["dy"] = torch.randn(T, n, generator=g, device=dev).to(dt)
    s["v"] = None
    if case["save_v"]:  # as the forward left it: A x of the rows before they were saved in 8 bits
        s["v"] = torch.zeros(T, _pad(max(ranks), 8), device=dev)
        for a, r in enumerate(ranks):
            mine = (s["ids"] == a)[:, None]
            s["v"][:, :r] = torch.where(mine, x.to(dt).float() @ s["A"][a].float().t(), s["v"][:, :r])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    dev, T, dt = torch.device("cuda"), case["rows"], s["dtype"]
    if case["op"] == "save":
        ld = _pad(case["d"], BLOCK)
        s["codes"] = torch.zeros(T, ld, device=dev, dtype=torch.uint8)
        s["scales"] = torch.full((T, _pad(ld // BLOCK, 4)), 127, device=dev, dtype=torch.uint8)
    elif case["op"] == "restore":
        s["x"] = torch.empty(T, case["d"], device=dev, dtype=dt)
    elif case["op"] == "base":
        s["out"] = torch.empty(T, case["d_out"], device=dev, dtype=dt)
    else:
        # the gradients of all adapters lie in one buffer, so that one fill clears them before a step
        shapes = [a.shape for a in s["A"]] + [b.shape for b in s["B"]]
        flat = torch.zeros(sum(v.numel() for v in shapes), device=dev)
        parts = [p.view(v) for p, v in zip(flat.split([v.numel() for v in shapes]), shapes)]
        s["grads"], s["dA"], s["dB"] = flat, parts[: len(s["A"])], parts[len(s["A"]):]
        s["dx"] = torch.empty(T, case["d_in"], device=dev, dtype=dt) if case["dx"] else None
        # which adapter and which rank each column of the concatenated factors belongs to
        s["owner"] = torch.repeat_interleave(torch.arange(len(s["ranks"]), device=dev), torch.tensor(s["ranks"], device=dev))
        s["rank"] = torch.cat([torch.arange(r, device=dev) for r in s["ranks"]])
        s["rate"] = torch.tensor(s["rates"], device=dev)[s["owner"]]
    if own:
        # what a program keeps: the views of the saved rows and the weight, the adapter tables,
        # the rows' grouping by adapter, the workspaces
        import expand_token_adapter_amd as lb

        d = case["d"] if "d" in case else case["d_in"]
        s["rows"] = lb.QuantRows(s["codes"], s["scales"], d)
        if case["op"] == "base":
            s["weight"] = lb.QuantWeight(s["wcodes"], s["wscales"], case["d_out"], d)
            s["ws"] = torch.empty(lb.lora_base_product_workspace_bytes(T, d, case["d_out"]), device=dev, dtype=torch.uint8)
        elif case["op"] == "backward":
            s["table"] = lb.AdapterTable(s["A"], s["B"], s["rates"])
            s["gtable"] = lb.GradTable(s["dA"], s["dB"])
            s["seg"] = lb.lora_segments_build(s["ids"], len(s["ranks"]))
            s["ws"] = torch.empty(lb.lora_backward_quant_workspace_bytes(dt, T, d, case["d_out"], max(s["ranks"])),
                                  device=dev, dtype=torch.uint8)
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    op = s["case"]["op"]
    if own:
        import expand_token_adapter_amd as lb

        if op == "save":
            lb.lora_quant_rows(s["x"], out=s["rows"])
            return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}
        if op == "restore":
            return lb.lora_dequant_rows(s["rows"], out=s["x"])
        if op == "base":
            if s["y"] is not None:
                s["out"].copy_(s["y"])  # the call adds to what is there
            return lb.lora_base_product(s["rows"], s["weight"], y=s["out"], accumulate=s["y"] is not None, ws=s["ws"])
        s["grads"].zero_()
        if s["dx"] is not None:
            s["dx"].zero_()
        lb.lora_backward_quant(s["rows"], s["dy"], s["table"], s["gtable"], s["seg"], dx=s["dx"], v_saved=s["v"], ws=s["ws"])
        return {"dA": s["dA"], "dB": s["dB"], "dx": s["dx"]}

    if op == "save":
        codes, scales = _plain_save(s["x"])
        return {"codes": codes, "scales": scales}
    if op == "restore":
        return _plain_rows(s["codes"], s["scales"], s["case"]["d"]).to(s["dtype"])
    k, n = s["case"]["d_in"], s["case"]["d_out"]
    x = _plain_rows(s["codes"], s["scales"], k)
    if op == "base":
        y = x @ _plain_weight(s["wcodes"], s["wscales"], n, k).t()
        return (y if s["y"] is None else s["y"].float() + y).to(s["dtype"])
    # every adapter at once: products with the concatenated factors, masked to each row's own adapter
    A, B = torch.cat(s["A"]).float(), torch.cat(s["B"], 1).float()
    dy, mine = s["dy"].float(), s["ids"][:, None] == s["owner"]
    v = torch.where(mine, x @ A.t() if s["v"] is None else s["v"][:, s["rank"]], 0.0)
    g = torch.where(mine, dy @ B, 0.0)
    dA = (s["rate"][:, None] * (g.t() @ x)).split(s["ranks"])
    dB = (s["rate"] * (dy.t() @ v)).split(s["ranks"], 1)
    return {"dA": list(dA), "dB": list(dB), "dx": ((s["rate"] * g) @ A).to(s["dtype"]) if s["dx"] is not None else None}


# ---------------------------------------------------------------- the definition, in 64 bits


def _exact_values(codes, scales, rows_per_scale):
    """code * 2^(scale - 127), decoded bit by bit: sign, 4 exponent bits (bias 7), 3 bits of fraction."""
    c = codes.int()
    e, f = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, torch.exp2(e.double() - 7) * (1 + f / 8), f / 512)
    row = torch.arange(c.shape[0], device=c.device) // rows_per_scale
    col = torch.arange(c.shape[1], device=c.device) // BLOCK
    return torch.where(c > 127, -mag, mag) * torch.exp2(scales.double() - 127)[row][:, col]


def exact(case, seed):
    s = _inputs(case, seed)
    T = case["rows"]
    if case["op"] == "save":
        d, nb = case["d"], -(-case["d"] // BLOCK)
        x = torch.nn.functional.pad(s["x"].double(), (0, nb * BLOCK - d)).view(T, nb, BLOCK)
        top = x.abs().amax(-1)
        e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp_min(1e-300) / 448)), 0.0).clamp(-127, 127)
        e = torch.where(top > 448 * torch.exp2(e), e + 1, e)  # (log2's own rounding)
        e = torch.where((top > 0) & (top <= 448 * torch.exp2(e - 1)) & (e > -127), e - 1, e)
        z = x / torch.exp2(e)[..., None]
        step = torch.exp2(torch.frexp(z)[1].double().clamp_min(-5) - 4)  # 4 significant bits, 2^-9 at the least
        scales = torch.full((T, _pad(nb, 4)), 127, device=x.device, dtype=torch.uint8)
        scales[:, :nb] = (e + 127).to(torch.uint8)
        return {"codes": (torch.round(z / step) * step).view(T, nb * BLOCK), "scales": scales}
    d = case["d"] if case["op"] == "restore" else case["d_in"]
    x = _exact_values(s["codes"], s["scales"], 1)[:, :d]
    if case["op"] == "restore":
        return x
    if case["op"] == "base":
        y = x @ _exact_values(s["wcodes"], s["wscales"], BLOCK)[:, :d].t()
        return y if s["y"] is None else y + s["y"].double()
    dA, dB, dx = [], [], torch.zeros(T, d, device=x.device, dtype=torch.float64)
    for a, (A, B, rate) in enumerate(zip(s["A"], s["B"], s["rates"])):
        A, B, at = A.double(), B.double(), torch.nonzero(s["ids"] == a)[:, 0]
        dy, xa = s["dy"][at].double(), x[at]
        g = dy @ B
        v = xa @ A.t() if s["v"] is None else s["v"][at, : A.shape[0]].double()
        dA.append(rate * (g.t() @ xa))
        dB.append(rate * (dy.t() @ v))
        dx[at] = rate * (g @ A)
    return {"dA": dA, "dB": dB, "dx": dx if case["dx"] else None}
