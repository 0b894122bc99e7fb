"""Limits of the 8-bit calls and of the calls beside them that hold without a GPU:
workspace sizes, refusals, and which kernels the tests' shapes reach."""
import math
import os
import random
import subprocess

import pytest
import torch

from expand_token_adapter_amd import _abi
from quant_plans import PRODUCTS

FAKE = 0x10000  # an aligned address that no check reads


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


# bytes that callers of lora_backward have kept since before the 8-bit calls
@pytest.mark.parametrize("args,want", [((0, 4096, 5120, 5120, 16), 16809984), ((0, 4096, 5120, 5120, 128), 39878656),
                                       ((0, 2048, 4096, 14336, 16), 18382848), ((0, 2048, 4096, 14336, 64), 27295744),
                                       ((1, 211, 1160, 776, 12), 10634752), ((0, 1, 8, 8, 1), 10519808)])
def test_backward_asks_for_no_more_than_it_did(lib, args, want):
    assert lib.lora_backward_workspace_bytes(*args) == want


def test_backward_sizes_hold_both_sets_of_partials_for_8_bit_rows(lib):
    """lora_backward_quant has room for g's and v's partials (one set each of slices of 512 columns) at once."""
    for T, d_in, d_out, r in ((4096, 5120, 5120, 128), (3000, 5120, 4096, 128), (8192, 14336, 512, 16), (64, 200, 512, 16)):
        both = (-(-d_in // 512) + -(-d_out // 512)) * T * r * 4
        assert lib.lora_backward_quant_workspace_bytes(0, T, d_in, d_out, r) >= both
        assert lib.lora_backward_quant_workspace_bytes(0, T, d_in, d_out, r) >= lib.lora_backward_workspace_bytes(0, T, d_in, d_out, r)


def _q(ld=128, lds=4):
    return _abi.LoraQuant(FAKE, ld, FAKE, lds)


@pytest.mark.parametrize("d,blocks", [(8, 1), (128, 1), (200, 2), (14336, 112)])
def test_rows_past_a_launch_are_refused(lib, d, blocks):
    """A launch has fewer than 2^32 threads, 8 (save) or 4 (restore) for a block of 128: more blocks are refused by
    the call, before a launch that would fail."""
    q = _q(ld=-(-d // 128) * 128, lds=blocks + -blocks % 4)
    pitch = -(-d // 8) * 8
    for limit, call in ((2 ** 29 - 32, lambda T: lib.lora_quant_rows(0, FAKE, pitch, T, d, q, None)),
                        (2 ** 30 - 64, lambda T: lib.lora_dequant_rows(0, q, T, d, FAKE, pitch, None))):
        T = limit // blocks + 1
        for t in (T, T + 1, 2 * T, 2 ** 31 - 1):
            assert call(min(t, 2 ** 31 - 1)) == _abi.LORA_ERR_UNSUPPORTED, t


def test_weights_past_a_launch_are_refused(lib):
    for d_out, d_in in ((8, 2 ** 31 - 8), (8, 2 ** 31 - 120), (128 * 65535 + 8, 8)):
        for tr in (0, 1):
            assert lib.lora_quant_weight(0, FAKE, d_in, d_out, d_in, tr, _q(ld=2 ** 31, lds=2 ** 25), None) == _abi.LORA_ERR_UNSUPPORTED


def test_any_slice_of_rows_is_rows(monkeypatch):
    """Rows inside wider buffers: a slice of one row or none has the width and pitch that its rows need, as longer
    slices have, and so has a weight of one row of scales."""
    import expand_token_adapter_amd as lb
    monkeypatch.setattr(lb, "_on_gpu", lambda *ts: None)
    codes, scales = torch.zeros(6, 640, dtype=torch.uint8)[:, :500], torch.zeros(6, 12, dtype=torch.uint8)[:, :5]
    q = lb.QuantRows(codes, scales, 300)
    assert (q.c.ld, q.c.lds) == (640, 12)
    for a, b in ((0, 6), (1, 3), (2, 3), (5, 6), (4, 4)):
        s = q[a:b]
        assert s.T == b - a and s.d == 300
        if s.T > 1:
            assert (s.c.ld, s.c.lds) == (640, 12)
        else:
            assert (s.c.ld, s.c.lds) == (384, 4)
        if s.T:
            assert (s.c.codes, s.c.scales) == (codes[a:].data_ptr(), scales[a:].data_ptr())
    w = lb.QuantWeight(codes, scales[:1], 6, 300)
    assert (w.c.ld, w.c.lds) == (640, 4)
    with pytest.raises(ValueError):
        lb.QuantRows(codes[:, :380], scales, 300)  # too narrow for three blocks
    with pytest.raises(ValueError):
        lb.QuantRows(torch.zeros(6, 500, dtype=torch.uint8), scales, 300)  # pitch 500
    with pytest.raises(ValueError):
        lb.QuantRows(codes[:1, :380], scales[:1], 300)


def test_backward_names_rows_of_the_wrong_form(monkeypatch):
    """8-bit rows given to the calls that take tensors, and a tensor to the one that takes 8-bit rows."""
    import expand_token_adapter_amd as lb
    monkeypatch.setattr(lb, "_on_gpu", lambda *ts: None)
    q = lb.QuantRows(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 8)
    dy, status = torch.zeros(4, 8), torch.zeros(1, dtype=torch.int32)

    class Table:  # of adapters 8 -> 8, as far as the checks before x's read it
        device, d_in, d_out, dtype, r_max = torch.device("cpu"), 8, 8, torch.bfloat16, 8

        def __len__(self):
            return 1

    with pytest.raises(TypeError, match="lora_backward_quant"):
        lb.lora_backward(q, dy, Table(), None, None)
    with pytest.raises(TypeError, match="lora_backward_quant"):
        lb._backward("lora_backward_preemptible", q, dy, Table(), None, None, None, None, None, None, (0, status.data_ptr()))
    with pytest.raises(TypeError, match="QuantRows"):
        lb.lora_backward_quant(torch.zeros(4, 8), dy, Table(), None, None)


# ---------------------------------------------------------------- which kernel a product takes

PLAN = """
#include <stdio.h>
#include "base_plan.h"
using namespace lora;
template <int K>
int piece() { return 4 * BaseLds<kTiles[K].bn, kTiles[K].bt, kTiles[K].stages>::kGroups; }
int main() {
    const int pieces[kKinds] = {INT32_MAX, piece<1>(), piece<2>(), piece<3>(), piece<4>(), piece<5>(), piece<6>()};
    long dt, T, k, n;
    while (scanf("%ld %ld %ld %ld", &dt, &T, &k, &n) == 4) {
        const BasePlan b = base_plan((int)dt, T, k, n);
        if (b.kind == kKinds) {
            printf("none 1 1 %zu\\n", base_workspace_bytes(b, T, n));
            continue;
        }
        const long nkb = (k + 127) / 128, groups = (nkb + 3) / 4, part = (groups + b.splits - 1) / b.splits * 4;
        const long most = part < nkb ? part : nkb;
        const BaseTile& c = kTiles[b.kind];
        printf("%dx%d %d %ld %zu\\n", c.bn, c.bt, b.splits, (most + pieces[b.kind] - 1) / pieces[b.kind],
               base_workspace_bytes(b, T, n));
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """(type, rows, k, outputs) of each product -> (tile, parts of k, pieces of a part, workspace bytes)."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PLAN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(root, "include"), "-I",
                    os.path.join(root, "expand_token_adapter_amd", "csrc"), str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def ask(sizes):
        text = "".join(f"{int(dt == 'f32')} {T} {k} {n}\n" for dt, T, k, n in sizes)
        out = subprocess.run([str(d / "plan")], input=text, check=True, capture_output=True, text=True).stdout.split("\n")
        return [(t.replace("0x0", "stream"), int(s), int(p), int(w)) for t, s, p, w in (l.split() for l in out if l)]

    return ask


def test_listed_products_take_the_kernels_they_are_listed_for(plan):
    got = plan([s[:4] for s in PRODUCTS])
    assert [(*s[:4], *g[:3]) for s, g in zip(PRODUCTS, got)] == PRODUCTS


def test_listed_products_take_every_kernel(plan, lib):
    """Nothing that the choice reaches is left out of the list: 40 000 sizes over the whole range."""
    listed = {(s[0], s[4], s[5] > 1, s[6] > 1) for s in PRODUCTS}
    rng = random.Random(1)
    log = lambda lo, hi: int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    sizes = [(rng.choice(["bf16", "f32"]), log(1, 10000), 8 * log(1, 16000), 8 * log(1, 8000)) for _ in range(40000)]
    got = plan(sizes)
    assert {(s[0], g[0], g[1] > 1, g[2] > 1) for s, g in zip(sizes, got)} <= listed
    for s, g in zip(sizes[:500], got):
        assert g[3] <= lib.lora_base_product_workspace_bytes(*s[1:])


def _threads(tile, parts, T, n):
    bn, bt = (16, 1 << 31) if tile == "stream" else map(int, tile.split("x"))
    return (-(-n // bn) * -(-T // bt) * parts + 7) * (512 if tile in ("stream", "256x256") else 256)


def test_products_of_very_many_rows_or_outputs_fit_a_launch(plan, lib):
    """The choice passes over kernels whose launch would have 2^32 threads or more; what none holds is refused before
    a launch that would fail."""
    rows, outputs = [2 ** 20, 2 ** 26, 2 ** 30, 2 ** 30 + 64, 2 ** 31 - 264], [8, 128, 2 ** 20, 2 ** 27, 2 ** 27 + 8, 2 ** 31 - 264]
    sizes = [(dt, T, k, n) for dt in ("bf16", "f32") for k in (8, 128, 4096) for T in [1, 3, 16, 17, 300] + rows
             for n in outputs] + [(dt, T, k, n) for dt in ("bf16", "f32") for k in (8, 128, 4096) for T in rows for n in outputs[:3]]
    for (dt, T, k, n), (tile, parts, _, need) in zip(sizes, plan(sizes)):
        if tile != "none":
            assert _threads(tile, parts, T, n) < 2 ** 32, (dt, T, k, n, tile)
        else:
            assert (T + n) * -(-k // 128) * 128 + T * n * (4 if dt == "f32" else 2) > 288e9  # more than a GPU holds
            q = _q(ld=4096, lds=32)
            assert lib.lora_base_product(int(dt == "f32"), q, T, k, q, n, FAKE, n, 0, FAKE, 2 ** 62, None) == _abi.LORA_ERR_UNSUPPORTED
            assert need == 16
