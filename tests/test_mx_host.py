"""Refusals of the 4-bit and expert calls, before anything touches the GPU: the library's own checks (through its C
ABI, with addresses that are never read) and the binding's; the choice of kernel and its workspace; the oracle of
the form."""
import numpy as np
import pytest
import torch

import mx_helpers as mh
from expand_token_adapter_amd import ExpertSegments, MxRows, MxWeight, _abi
import expand_token_adapter_amd as lb

FAKE = 0x10000
BAD, UNS, WS, OK = _abi.LORA_ERR_INVALID_ARG, _abi.LORA_ERR_UNSUPPORTED, _abi.LORA_ERR_WORKSPACE, _abi.LORA_OK


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


def _q(codes=FAKE, ld=256, scales=FAKE, lds=16):  # 300 columns: 2 units of 256
    return _abi.LoraQuant(codes, ld, scales, lds)


def _seg():
    return _abi.LoraSegments(FAKE, FAKE, FAKE, FAKE, FAKE)


BAD_MX = [(dict(codes=None), BAD), (dict(codes=FAKE + 8), BAD), (dict(scales=None), BAD), (dict(scales=FAKE + 4), BAD),
          (dict(ld=128), BAD), (dict(ld=320), UNS), (dict(lds=8), BAD), (dict(lds=20), UNS)]


@pytest.mark.parametrize("fn", ["lora_quant_rows_mx", "lora_dequant_rows_mx"])
def test_rows_refusals(lib, fn):
    def call(dtype=0, x=FAKE, ldx=304, T=4, d=304, q=None):
        q = q or _q()
        if fn == "lora_quant_rows_mx":
            return lib.lora_quant_rows_mx(dtype, x, ldx, T, d, q, None)
        return lib.lora_dequant_rows_mx(dtype, q, T, d, x, ldx, None)

    assert call(T=0, x=None) == OK
    assert call(dtype=2) == BAD and call(T=-1) == BAD and call(d=0) == BAD
    assert call(x=None) == BAD and call(x=FAKE + 4) == BAD and call(ldx=296) == BAD
    assert call(d=300) == UNS and call(ldx=308) == UNS
    assert call(T=2 ** 29) == UNS  # 2^30 units
    for kw, want in BAD_MX:
        assert call(q=_q(**kw)) == want, kw


def test_weight_refusals(lib):
    def call(dtype=0, w=FAKE, ldw=304, n=264, k=304, tr=0, q=None):
        return lib.lora_quant_weight_mx(dtype, w, ldw, n, k, tr, q or _q(), None)

    assert call(dtype=3) == BAD and call(n=0) == BAD and call(k=0) == BAD and call(tr=2) == BAD
    assert call(w=None) == BAD and call(ldw=128) == BAD
    assert call(n=260) == UNS and call(k=300) == UNS
    for kw, want in BAD_MX:
        assert call(q=_q(**kw)) == want, kw
        assert call(tr=1, q=_q(**kw)) == want, kw
    assert call(n=2 ** 23 + 8) == UNS and call(tr=1, k=2 ** 23 + 8, ldw=2 ** 23 + 8) == UNS


def _q8():
    return _abi.LoraQuant(FAKE, 384, FAKE, 4)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("experts", [None, 4])
def test_product_refusals(lib, bits, experts):
    need = lib.lora_base_product_mx_workspace_bytes(4, 304, 136)
    rows = _q() if bits == 4 else _q8()

    def call(dtype=0, bits=bits, x=None, T=4, k=304, w=None, n=136, y=FAKE, ldy=136, add=0, ws=FAKE, nb=need, E=experts, seg=None):
        if experts is None:
            return lib.lora_base_product_mx(dtype, bits, x or rows, T, k, w or _q(), n, y, ldy, add, ws, nb, None)
        return lib.lora_expert_product_mx(dtype, bits, x or rows, T, k, w or _q(), E, n, seg or _seg(), y, ldy, add, None)

    assert call(T=0, y=None, ws=None, nb=0) == OK
    assert call(dtype=-1) == BAD and call(T=-1) == BAD and call(k=0) == BAD and call(n=0) == BAD and call(add=2) == BAD
    assert call(bits=5) == BAD and call(bits=16) == BAD
    assert call(y=None) == BAD and call(y=FAKE + 2) == BAD and call(ldy=128) == BAD
    assert call(k=300) == UNS and call(n=132, ldy=136) == UNS and call(ldy=140) == UNS
    for kw, want in BAD_MX:
        assert call(w=_q(**kw)) == want, kw
        if bits == 4:
            assert call(x=_q(**kw)) == want, kw
    if bits == 8:
        assert call(x=_abi.LoraQuant(FAKE, 256, FAKE, 4)) == BAD and call(x=_abi.LoraQuant(FAKE, 384, FAKE, 6)) == UNS
    huge = (1 << 22) + 128
    for kw in (dict(ld=huge), dict(lds=huge)):
        assert call(w=_q(**kw)) == UNS
        assert call(x=_q(**kw) if bits == 4 else _abi.LoraQuant(FAKE, kw.get("ld", 384), FAKE, kw.get("lds", 4))) == UNS
    assert call(T=2 ** 31 - 1, nb=2 ** 62) == UNS and call(n=2 ** 31 - 8, ldy=2 ** 31, nb=2 ** 62) == UNS
    if experts is None:
        assert call(nb=need - 1) == WS and call(ws=None) == WS and call(ws=FAKE + 8) == WS
    else:
        assert call(E=0) == BAD and call(seg=_abi.LoraSegments(FAKE, None, FAKE, FAKE, FAKE)) == BAD


def test_expert_segments_refusals(lib):
    need = lib.lora_segments_workspace_bytes(100, 4)

    def call(ids=FAKE, T=50, k=2, E=4, seg=None, pos=FAKE, ws=FAKE, nb=need):
        return lib.lora_expert_segments(ids, T, k, E, seg or _seg(), pos, ws, nb, None)

    assert call(T=0, ids=None, pos=None, ws=None, nb=0) == OK
    assert call(T=-1) == BAD and call(k=0) == BAD and call(E=0) == BAD and call(ids=None) == BAD
    assert call(pos=None) == BAD and call(pos=FAKE + 2) == BAD
    assert call(seg=_abi.LoraSegments(FAKE, FAKE, FAKE, FAKE, None)) == BAD
    assert call(nb=need - 1) == WS and call(ws=None) == WS
    assert call(T=2 ** 30, k=2, nb=2 ** 62) == BAD  # 2^31 choices


@pytest.mark.parametrize("fn", ["gather", "gather_backward", "combine", "combine_backward"])
def test_row_movement_refusals(lib, fn):
    def call(dtype=0, a=FAKE, lda=64, T=5, d=64, k=2, pos=FAKE, w=FAKE, b=FAKE, ldb=64, add=0):
        """a: what is read, b: what is written"""
        if fn == "gather":
            return lib.lora_expert_gather(dtype, a, lda, T, d, k, pos, b, ldb, None)
        if fn == "gather_backward":
            return lib.lora_expert_gather_backward(dtype, a, lda, T, d, k, pos, b, ldb, add, None)
        if fn == "combine":
            return lib.lora_expert_combine(dtype, a, lda, T, d, k, pos, w, b, ldb, add, None)
        return lib.lora_expert_combine_backward(dtype, a, lda, FAKE, max(lda, 64), T, d, k, pos, w, b, ldb, FAKE, None)

    assert call(T=0, a=None, b=None, pos=None, w=None) == OK
    assert call(dtype=2) == BAD and call(T=-1) == BAD and call(d=0) == BAD and call(k=0) == BAD
    assert call(pos=None) == BAD and call(pos=FAKE + 1) == BAD
    assert call(T=2 ** 30, k=2) == BAD
    assert call(a=None) == BAD and call(a=FAKE + 8) == BAD and call(lda=56) == BAD and call(lda=68) == UNS
    assert call(b=FAKE + 8) == BAD and call(ldb=56) == BAD and call(ldb=68) == UNS
    assert call(d=60) == UNS
    assert call(T=2 ** 30, k=1, d=2 ** 12, lda=2 ** 12, ldb=2 ** 12) == UNS  # more threads than a launch has
    if fn != "combine_backward":
        assert call(b=None) == BAD
    if fn.startswith("combine"):
        assert call(w=None) == BAD and call(w=FAKE + 2) == BAD
    if fn in ("gather_backward", "combine"):
        assert call(add=2) == BAD


def test_combine_backward_optional_outputs(lib):
    def call(o=FAKE, d_o=FAKE, dw=FAKE):
        return lib.lora_expert_combine_backward(0, FAKE, 64, o, 64, 5, 68, 2, FAKE, FAKE, d_o, 64, dw, None)

    assert call(d_o=None, dw=None) == BAD and call(dw=FAKE + 2) == BAD  # nothing to compute; bad alignment
    assert lib.lora_expert_combine_backward(0, FAKE, 64, None, 0, 5, 64, 2, FAKE, FAKE, FAKE, 64, FAKE, None) == BAD  # dw needs o


def test_queries_and_plans(lib):
    ask = lib.lora_base_product_mx_workspace_bytes
    assert ask(-1, 8, 8) == 0 and ask(1, 0, 8) == 0 and ask(1, 8, 0) == 0 and ask(0, 8, 8) == 16
    rng = np.random.default_rng(3)
    for T, k, n in np.exp(rng.uniform(0, np.log(1 << 20), size=(4000, 3))).astype(int) + 1:
        assert 16 <= ask(int(T), 8 * int(k), 8 * int(n)) <= lb.LORA_BASE_PRODUCT_MAX_WORKSPACE
    for T in range(1, 3000):
        assert ask(T, 14336, 4096) <= lb.LORA_BASE_PRODUCT_MAX_WORKSPACE


def test_binding_refuses():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    with pytest.raises(ValueError):
        MxRows(u8(4, 128), u8(4, 8), 200)  # not on the GPU
    with pytest.raises(TypeError):
        MxRows(torch.zeros(4, 128), u8(4, 8), 200)
    with pytest.raises(TypeError):
        MxWeight(u8(4, 128), torch.zeros(4, 8), 4, 200)
    with pytest.raises(ValueError):
        MxWeight(u8(4, 128), u8(4, 8), 4, 200, experts=0)
    for call in (lb.lora_quant_rows_mx, lb.lora_quant_weight_mx):
        with pytest.raises(ValueError):
            call(torch.zeros(4, 8))
    with pytest.raises(TypeError):
        lb.lora_dequant_rows_mx(torch.zeros(4, 8))
    with pytest.raises(TypeError):
        lb.lora_base_product_mx(torch.zeros(4, 8), torch.zeros(4, 8))
    with pytest.raises(TypeError):
        lb.lora_expert_product_mx(torch.zeros(4, 8), torch.zeros(4, 8), None)
    with pytest.raises(ValueError):
        lb.lora_expert_segments(torch.zeros(4, 2, dtype=torch.int32), 4)
    for call in (lambda: lb.lora_expert_gather(torch.zeros(4, 8), None), lambda: lb.lora_expert_gather_backward(torch.zeros(8, 8), None),
                 lambda: lb.lora_expert_combine(torch.zeros(8, 8), torch.zeros(4, 2), None),
                 lambda: lb.lora_expert_combine_backward(torch.zeros(4, 8), torch.zeros(8, 8), torch.zeros(4, 2), None)):
        with pytest.raises(TypeError):
            call()
    seg = ExpertSegments(4, 2, 3, torch.device("cpu"))
    assert seg.T == 8 and seg.num_adapters == 3 and seg.pos.shape == (4, 2)
    with pytest.raises(ValueError):
        lb.lora_expert_gather(torch.zeros(4, 8), seg)  # not on the GPU


def test_the_oracle_of_the_form():
    assert list(mh.E2M1[:8]) == [0, 0.5, 1, 1.5, 2, 3, 4, 6] and list(mh.E2M1[8:]) == [-v for v in mh.E2M1[:8]]
    z = np.array([0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 6.0, -0.25, -5.0])
    assert list(mh.E2M1[mh.encode_codes(z)]) == [0, 0.5, 1, 1, 2, 2, 3, 4, 4, 6, 6, 0, -4]
    assert list(mh.scale_bytes(np.array([6.0, 6.01, 3.0, 1.5, 1.51, 0.0, 1e-45, np.inf]))) == [127, 128, 126, 125, 126, 127, 0, 255]
    a = np.random.default_rng(1).standard_normal((70, 300))
    for square in (False, True):
        c, s = mh.quant(a, square)
        assert c.shape == (70, 512) and s.shape == (70, 16) and np.array_equal(mh.unpack(mh.pack(c)), c)
        v = mh.values(c, s, 300)
        # half a step: 0.25 below 2, a quarter of the power of two above, of a scale at most 2 * max / 6
        assert np.all(np.abs(v - a) <= np.maximum(0.25 * mh.expand(s, 32, 300), 2.0 ** -2 * np.abs(a)))
    ct, st = mh.quant(a.T, True)
    c, s = mh.quant(a, True)
    assert np.array_equal(mh.values(ct, st, 70).T, mh.values(c, s, 300))
    ids = np.array([[1, 0], [-1, 1], [1, 2]])
    off, perm, pos = mh.sort_choices(ids, 4)
    assert list(off) == [0, 1, 4, 5, 5] and list(perm) == [1, 0, 3, 4, 5] and pos.tolist() == [[1, 0], [-1, 2], [3, 4]]
