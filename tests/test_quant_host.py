"""Refusals of the 8-bit calls, before anything touches the GPU: the library's
own checks (through its C ABI, with addresses that are never read) and the
binding's."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

import quant_helpers as qh
from expand_token_adapter_amd import QuantRows, QuantWeight, _abi
import expand_token_adapter_amd as lb

FAKE = 0x10000
BAD, UNS, WS, OK = _abi.LORA_ERR_INVALID_ARG, _abi.LORA_ERR_UNSUPPORTED, _abi.LORA_ERR_WORKSPACE, _abi.LORA_OK


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


def _q(codes=FAKE, ld=256, scales=FAKE, lds=4):
    return _abi.LoraQuant(codes, ld, scales, lds)


def _seg():
    return _abi.LoraSegments(FAKE, FAKE, FAKE, FAKE, FAKE)


BAD_QUANT = [(dict(codes=None), BAD), (dict(codes=FAKE + 8), BAD), (dict(scales=None), BAD), (dict(scales=FAKE + 2), BAD),
             (dict(ld=128), BAD), (dict(ld=320), UNS), (dict(lds=1), BAD), (dict(lds=5), UNS)]  # 200 columns: 2 blocks


def test_struct_matches_header(tmp_path):
    import os
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    src = tmp_path / "p.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "lora_batch.h"\nint main(void) { printf("%zu %zu %zu %d", '
                   'sizeof(lora_quant), offsetof(lora_quant, scales), offsetof(lora_quant, lds), LORA_QUANT_BLOCK); return 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-I", inc, str(src), "-o", str(tmp_path / "p")], check=True)
    got = subprocess.run([str(tmp_path / "p")], check=True, capture_output=True, text=True).stdout.split()
    q = _abi.LoraQuant
    assert [int(v) for v in got] == [ctypes.sizeof(q), q.scales.offset, q.lds.offset, _abi.LORA_QUANT_BLOCK]


@pytest.mark.parametrize("fn", ["lora_quant_rows", "lora_dequant_rows"])
def test_rows_refusals(lib, fn):
    def call(dtype=0, x=FAKE, ldx=200, T=4, d=200, q=None):
        q = q or _q()
        if fn == "lora_quant_rows":
            return lib.lora_quant_rows(dtype, x, ldx, T, d, q, None)
        return lib.lora_dequant_rows(dtype, q, T, d, x, ldx, None)

    assert call(T=0, x=None) == OK
    assert call(dtype=2) == BAD and call(T=-1) == BAD and call(d=0) == BAD
    assert call(x=None) == BAD and call(x=FAKE + 4) == BAD and call(ldx=192) == BAD
    assert call(d=196) == UNS and call(ldx=204) == UNS
    assert call(T=2 ** 30) == UNS  # 2^31 blocks
    for kw, want in BAD_QUANT:
        assert call(q=_q(**kw)) == want, kw


def test_weight_refusals(lib):
    def call(dtype=0, w=FAKE, ldw=200, n=136, k=200, tr=0, q=None):
        return lib.lora_quant_weight(dtype, w, ldw, n, k, tr, q or _q(), None)

    assert call(dtype=3) == BAD and call(n=0) == BAD and call(k=0) == BAD and call(tr=2) == BAD
    assert call(w=None) == BAD and call(ldw=128) == BAD
    assert call(n=132) == UNS and call(k=196) == UNS
    for kw, want in BAD_QUANT:
        assert call(q=_q(**kw)) == want, kw
    assert call(tr=1, q=_q(ld=128)) == BAD  # the transposed rows have 136 columns


def test_base_product_refusals(lib):
    need = lib.lora_base_product_workspace_bytes(4, 200, 136)

    def call(dtype=0, x=None, T=4, k=200, w=None, n=136, y=FAKE, ldy=136, add=0, ws=FAKE, nb=need):
        return lib.lora_base_product(dtype, x or _q(), T, k, w or _q(), n, y, ldy, add, ws, nb, None)

    assert call(T=0, y=None, ws=None, nb=0) == OK
    assert call(dtype=-1) == BAD and call(T=-1) == BAD and call(k=0) == BAD and call(n=0) == BAD and call(add=2) == BAD
    assert call(y=None) == BAD and call(y=FAKE + 2) == BAD and call(ldy=128) == BAD
    assert call(k=196) == UNS and call(n=132, ldy=136) == UNS and call(ldy=140) == UNS
    for kw, want in BAD_QUANT:
        assert call(x=_q(**kw)) == want and call(w=_q(**kw)) == want, kw
    huge = (1 << 22) + 128
    assert call(x=_q(ld=huge)) == UNS and call(w=_q(ld=huge)) == UNS
    assert call(T=2 ** 31 - 1, nb=2 ** 62) == UNS and call(n=2 ** 31 - 8, ldy=2 ** 31, nb=2 ** 62) == UNS
    assert call(nb=need - 1) == WS and call(ws=None) == WS and call(ws=FAKE + 8) == WS


def test_backward_refusals(lib):
    need = lib.lora_backward_quant_workspace_bytes(0, 64, 200, 512, 16)
    assert need == lib.lora_backward_workspace_bytes(0, 64, 200, 512, 16) > 0

    def call(x=None, dtype=0, dy=FAKE, lddy=512, dx=None, T=64, k=200, A=4, r=16, v=None, ldv=0, ws=FAKE, nb=need):
        return lib.lora_backward_quant(dtype, x or _q(), dy, lddy, dx, 200, T, k, 512, FAKE, FAKE, A, r, _seg(), v, ldv,
                                       ws, nb, None)

    assert call(T=0, ws=None, nb=0) == OK
    for kw, want in BAD_QUANT:
        assert call(x=_q(**kw)) == want, kw
    assert call(dtype=2) == BAD and call(A=0) == BAD and call(r=129) == BAD and call(dy=None) == BAD
    assert call(lddy=504) == BAD and call(dx=FAKE + 4) == BAD and call(v=FAKE, ldv=8) == BAD and call(k=196) == UNS
    assert call(nb=need - 1) == WS


def test_queries(lib):
    assert lib.lora_base_product_workspace_bytes(-1, 8, 8) == 0 and lib.lora_base_product_workspace_bytes(1, 0, 8) == 0
    assert lib.lora_base_product_workspace_bytes(1, 8, 0) == 0 and lib.lora_base_product_workspace_bytes(0, 8, 8) > 0
    assert lib.lora_backward_quant_workspace_bytes(0, -1, 8, 8, 8) == 0
    # (parts of a split contraction: never more than a few tiles' worth for each CU)
    for T in (1, 16, 17, 300, 5000, 2 ** 31 - 1):
        for k in (8, 4096, 2 ** 22):
            for n in (8, 1032, 2 ** 20):
                assert 16 <= lib.lora_base_product_workspace_bytes(T, k, n) <= 256 * 256 * 256 * 4


def test_binding_refuses():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    with pytest.raises(ValueError):
        QuantRows(u8(4, 256), u8(4, 4), 200)  # not on the GPU
    with pytest.raises(TypeError):
        QuantRows(torch.zeros(4, 256), u8(4, 4), 200)
    with pytest.raises(TypeError):
        QuantWeight(u8(4, 256), torch.zeros(1, 4), 4, 200)
    with pytest.raises(ValueError):
        lb.lora_quant_rows(torch.zeros(4, 8))
    with pytest.raises(ValueError):
        lb.lora_quant_weight(torch.zeros(4, 8))
    with pytest.raises(TypeError):
        lb.lora_base_product(torch.zeros(4, 8), torch.zeros(4, 8))
    with pytest.raises(TypeError):
        lb.lora_backward_quant(torch.zeros(4, 8), None, None, None, None)


def test_the_oracle_of_the_form():
    """The tests' own 64-bit form: codes against torch's conversion, scales against their definition."""
    z = np.concatenate([np.random.default_rng(0).uniform(-448, 448, 4000), qh.E4M3[:127], (qh.E4M3[:126] + qh.E4M3[1:127]) / 2])
    t = torch.from_numpy(z).to(torch.float32).to(torch.float8_e4m3fn)
    assert np.array_equal(qh.encode_codes(z.astype(np.float32)), t.view(torch.uint8).numpy())
    assert np.array_equal(np.nan_to_num(qh.E4M3), torch.nan_to_num(torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()).numpy())
    top = np.array([448.0, 448.1, 224.0, 1.75, 1.76, 0.0, 1e-45])
    assert list(qh.scale_bytes(top)) == [127, 128, 126, 119, 120, 127, 0]
    a = np.random.default_rng(1).standard_normal((300, 200))
    c, s = qh.quant(a, 128)
    assert c.shape == (300, 256) and s.shape == (3, 2)
    v = qh.values(c, s, 200, 128)
    assert np.all(np.abs(v - a) <= 2.0 ** -4 * np.abs(a) + 2.0 ** -10 * 2.0 ** (s.max() - 127.0))  # half a step of 4 bits


def test_base_product_workspace_stays_below_its_bound():
    rng = np.random.default_rng(2)
    limit = lb.LORA_BASE_PRODUCT_MAX_WORKSPACE
    sizes = np.exp(rng.uniform(0, np.log(1 << 20), size=(4000, 3))).astype(int) + 1
    need = [lb.lora_base_product_workspace_bytes(int(T), 8 * int(k), 8 * int(n)) for T, k, n in sizes]
    assert max(need) <= limit and min(need) >= 16
    for T in range(1, 3000):  # every row count of a serving batch, one long k
        assert lb.lora_base_product_workspace_bytes(T, 14336, 4096) <= limit
