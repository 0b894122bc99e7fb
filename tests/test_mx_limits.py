"""Limits of the 4-bit and expert calls that hold without a GPU: refusals of what a launch does not hold, workspace
sizes, and which kernels the tests' shapes reach."""
import math
import os
import random
import subprocess

import pytest
import torch

from expand_token_adapter_amd import _abi
from mx_plans import EXPERTS, PRODUCTS

FAKE = 0x10000  # an aligned address that no check reads


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


def _q(ld, lds):
    return _abi.LoraQuant(FAKE, ld, FAKE, lds)


@pytest.mark.parametrize("d,units", [(8, 1), (256, 1), (304, 2), (14336, 56)])
def test_rows_past_a_launch_are_refused(lib, d, units):
    """A launch has fewer than 2^32 threads, 8 for a unit of 256 columns (fp32 restore: 16)."""
    q = _q(units * 128, units * 8)
    for limit, call in ((2 ** 29 - 64, lambda T: lib.lora_quant_rows_mx(0, FAKE, d, T, d, q, None)),
                        (2 ** 29 - 64, lambda T: lib.lora_quant_rows_mx(1, FAKE, d, T, d, q, None)),
                        (2 ** 29 - 64, lambda T: lib.lora_dequant_rows_mx(0, q, T, d, FAKE, d, None)),
                        (2 ** 28 - 32, lambda T: lib.lora_dequant_rows_mx(1, q, T, d, FAKE, d, None))):
        T = limit // units + 64 // units + 1
        for t in (T, T + 1, 2 * T, 2 ** 31 - 1):
            assert call(min(t, 2 ** 31 - 1)) == _abi.LORA_ERR_UNSUPPORTED, t


def test_weights_past_a_launch_are_refused(lib):
    for tr, d_out, d_in in ((0, 128 * 65535 + 8, 8), (1, 8, 128 * 65535 + 8)):
        assert lib.lora_quant_weight_mx(0, FAKE, d_in, d_out, d_in, tr, _q(2 ** 31, 2 ** 26), None) == _abi.LORA_ERR_UNSUPPORTED


def test_any_slice_of_rows_is_rows(monkeypatch):
    import expand_token_adapter_amd as lb
    monkeypatch.setattr(lb, "_on_gpu", lambda *ts: None)
    codes, scales = torch.zeros(6, 384, dtype=torch.uint8)[:, :300], torch.zeros(6, 24, dtype=torch.uint8)[:, :17]
    q = lb.MxRows(codes, scales, 300)
    assert (q.c.ld, q.c.lds) == (384, 24)
    for a, b in ((0, 6), (1, 3), (2, 3), (5, 6), (4, 4)):
        s = q[a:b]
        assert s.T == b - a and s.d == 300
        assert (s.c.ld, s.c.lds) == ((384, 24) if s.T > 1 else (256, 16))
        if s.T:
            assert (s.c.codes, s.c.scales) == (codes[a:].data_ptr(), scales[a:].data_ptr())
    w = q.as_weight(3)
    assert (w.d_out, w.d_in, w.experts) == (2, 300, 3) and w.rows().T == 6 and q.as_weight().experts is None
    for bad in (lambda: q.as_weight(4), lambda: lb.MxRows(codes[:, :250], scales, 300), lambda: lb.MxRows(codes, scales[:, :15], 300),
                lambda: lb.MxRows(torch.zeros(6, 300, dtype=torch.uint8), scales, 300), lambda: lb.MxRows(codes, scales[:5], 300),
                lambda: lb.MxWeight(codes, scales, 5, 300)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q[0], lambda: q[::2]):
        with pytest.raises(TypeError):
            bad()


# ---------------------------------------------------------------- which kernel a product takes

PLAN = """
#include <stdio.h>
#include "mx_plan.h"
using namespace lora;
template <int K>
constexpr bool lds() {
    constexpr MxTile c = kMxTiles[K];
    return MxLds<c.bn, c.bt, c.stages4, 4>::kBytes <= kLdsBytes && MxLds<c.bn, c.bt, c.stages8, 8>::kBytes <= kLdsBytes;
}
static_assert(lds<kMx64x32>() && lds<kMx64x64>() && lds<kMx128x128>() && lds<kMx256x128>() && lds<kMx256x256>(), "a CU's LDS");
int main() {
    long bits, dt, T, k, n, e;
    while (scanf("%ld %ld %ld %ld %ld %ld", &bits, &dt, &T, &k, &n, &e) == 6) {
        int64_t tiles_t = 0;
        const BasePlan b = e ? mx_expert_plan((int)bits, (int)dt, T, k, n, e, &tiles_t) : mx_plan((int)bits, (int)dt, T, k, n);
        if (b.kind == kMxKinds) {
            printf("none 1 0 %zu 0\\n", base_workspace_bytes(b, T, n));
            continue;
        }
        const MxTile& c = kMxTiles[b.kind];
        printf("%dx%d %d %d %zu %ld\\n", c.bn, c.bt, b.splits, mx_waves(b.kind, (int)bits, (int)dt), base_workspace_bytes(b, T, n), (long)tiles_t);
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """(bits, type, rows, k, outputs, experts or 0) of each -> (tile, parts of k, waves, workspace bytes, most tiles along t)."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    d = tmp_path_factory.mktemp("mxplan")
    (d / "plan.cpp").write_text(PLAN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(root, "include"), "-I",
                    os.path.join(root, "expand_token_adapter_amd", "csrc"), str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def ask(sizes):
        text = "".join(f"{bits} {int(dt == 'f32')} {T} {k} {n} {e}\n" for bits, dt, T, k, n, e in sizes)
        out = subprocess.run([str(d / "plan")], input=text, check=True, capture_output=True, text=True).stdout.split("\n")
        return [(t, int(s), int(w), int(b), int(m)) for t, s, w, b, m in (l.split() for l in out if l)]

    return ask


def test_listed_sizes_take_the_kernels_they_are_listed_for(plan):
    got = plan([(*s[:5], 0) for s in PRODUCTS])
    assert [(*s[:5], *g[:2]) for s, g in zip(PRODUCTS, got)] == PRODUCTS
    got = plan([(*s[:3], *s[4:6], s[3]) for s in EXPERTS])
    assert [(*s[:6], g[0]) for s, g in zip(EXPERTS, got)] == EXPERTS


def test_listed_sizes_take_every_kernel(plan, lib):
    rng = random.Random(1)
    log = lambda lo, hi: int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    sizes = [(rng.choice([4, 8]), rng.choice(["bf16", "f32"]), log(1, 10000), 8 * log(1, 8000), 8 * log(1, 4000), rng.choice([0, log(1, 400)]))
             for _ in range(40000)]
    got = plan(sizes)
    listed = {(s[0], s[1], s[5], s[6] > 1) for s in PRODUCTS}
    assert {(s[0], s[1], g[0], g[1] > 1) for s, g in zip(sizes, got) if not s[5]} <= listed
    experts = {(s[0], s[1], s[6]) for s in EXPERTS}
    assert {(s[0], s[1], g[0]) for s, g in zip(sizes, got) if s[5]} <= experts
    for s, g in zip(sizes, got):
        bn, bt = map(int, g[0].split("x"))
        if s[5]:  # room for the rows however they are spread, and no split
            assert g[1] == 1 and g[4] >= -(-s[2] // bt) and g[4] >= min(s[2], s[5])
        else:
            assert g[3] <= lib.lora_base_product_mx_workspace_bytes(*s[2:5]) <= _abi.LORA_BASE_PRODUCT_MAX_WORKSPACE
            assert g[1] <= -(-s[3] // 1024)  # parts of whole spans of scales


def test_products_of_very_many_rows_or_outputs_fit_a_launch(plan, lib):
    rows, outputs = [2 ** 20, 2 ** 26, 2 ** 30, 2 ** 30 + 64, 2 ** 31 - 264], [8, 128, 2 ** 20, 2 ** 27, 2 ** 27 + 8, 2 ** 31 - 264]
    sizes = [(bits, dt, T, k, n, e) for bits in (4, 8) for dt in ("bf16", "f32") for k in (8, 4096) for T in [1, 3, 300] + rows for n in outputs
             for e in (0, 1, 100)]
    for (bits, dt, T, k, n, e), (tile, parts, waves, need, most) in zip(sizes, plan(sizes)):
        if tile != "none":
            bn, bt = map(int, tile.split("x"))
            tiles = -(-n // bn) * (most if e else -(-T // bt)) * parts
            assert (tiles + 7) * waves * 64 < 2 ** 32, (bits, dt, T, k, n, e, tile)
        else:
            x, w = _q(4096, 128), _q(4096, 128)
            if e:
                seg = _abi.LoraSegments(FAKE, FAKE, FAKE, FAKE, FAKE)
                got = lib.lora_expert_product_mx(int(dt == "f32"), bits, x, T, k, w, e, n, seg, FAKE, n, 0, None)
            else:
                got = lib.lora_base_product_mx(int(dt == "f32"), bits, x, T, k, w, n, FAKE, n, 0, FAKE, 2 ** 62, None)
            assert got == _abi.LORA_ERR_UNSUPPORTED
            held = T * n * (4 if dt == "f32" else 2) + (T * 132 + max(1, e) * n * 136) * -(-k // 256)
            many = bits == 8 and dt == "f32" and -(-n // 256) * -(-T // 128) >= 2 ** 23 - 8  # (tiles of 8 waves)
            assert many or held > 288e9  # more than a GPU holds


def test_weights_of_more_rows_than_a_launch_are_refused(lib):
    """The documented limits; one row more is refused before anything is enqueued."""
    for transpose, most in ((0, 128 * 65535), (1, 64 * 65535)):
        n, k = (8, most + 8) if transpose else (most + 8, 8)
        assert lib.lora_quant_weight_mx(0, FAKE, k, n, k, transpose, _q(128, 8), None) == _abi.LORA_ERR_UNSUPPORTED
