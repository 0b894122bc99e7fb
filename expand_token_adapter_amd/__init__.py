"""Multi-LoRA batched adapter kernels for AMD MI355X (gfx950).

Python binding of the C ABI (include/lora_batch.h).  Each function has the
name of the C entry point it calls, takes torch tensors that live on the GPU,
and only marshals pointers, sizes and the current HIP stream: every step of
the computation runs in the HIP kernels of liblora_batch.so.  PyTorch supplies
device memory and streams.

    seg = lora_segments_build(ids, num_adapters)         # group rows by adapter
    v = lora_shrink(x, table, seg)                       # v = A_a x    (fp32)
    lora_expand_add(v, table, seg, y)                    # y += s_a B_a v
    lora_backward(x_ft, dy, table, grads, seg_ft, dx)    # dX, dA, dB  (+=)

Rows and frozen weights in 8 bits (e4m3 codes, one power-of-two scale per
block of 128):

    xq = lora_quant_rows(x)                              # save the layer input
    wq, wt = lora_quant_weight(W), lora_quant_weight(W, transpose=True)
    y = lora_base_product(xq, wq)                        # y = W x
    lora_base_product(lora_quant_rows(dy), wt, y=dx)     # dX = W^T dY
    lora_backward_quant(xq[s:e], dy, table, grads, seg_ft, dx)   # dX, dA, dB from the saved rows

A frozen weight in microscaled 4 bits (e2m1 codes, one power-of-two scale per 32
columns), for rows in 8 or 4 bits:

    w4 = lora_quant_rows_mx(W).as_weight()               # forward alone: a scale for each row's 32 columns
    w4, wt4 = lora_quant_weight_mx(W), lora_quant_weight_mx(W, transpose=True)   # the same values in both
    y = lora_base_product_mx(xq, w4)                     # y = W x

A mixture of experts: every token's rows to its k experts and back:

    seg = lora_expert_segments(expert_ids, num_experts)  # [T, k] choices, sorted by expert
    rows = lora_expert_gather(x, seg)                    # [T k, d]
    out = lora_expert_product_mx(lora_quant_rows(rows), w4, seg)   # each expert's rows through its weight
    y = lora_expert_combine(out, router_weights, seg)    # y[t] = sum_j w[t, j] out[pos[t, j]]
    d_out, dw = lora_expert_combine_backward(dy, out, router_weights, seg)
    dx = lora_expert_gather_backward(d_rows, seg)
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _abi
from ._abi import LORA_BASE_PRODUCT_MAX_WORKSPACE, LORA_BF16, LORA_F32, LORA_MAX_RANK, LoraError

__all__ = [
    "AdapterTable", "GradTable", "QuantRows", "QuantWeight", "Segments", "LoraError",
    "lora_segments_build", "lora_segments_build_batch", "lora_shrink", "lora_shrink_noalloc", "lora_expand_add",
    "lora_forward",
    "lora_forward_multi", "lora_backward", "lora_backward_preemptible", "lora_adamw_step",
    "lora_quant_rows", "lora_dequant_rows", "lora_quant_weight", "lora_base_product", "lora_backward_quant",
    "lora_abi_version", "lora_status_string", "LORA_BASE_PRODUCT_MAX_WORKSPACE",
    "lora_segments_workspace_bytes", "lora_shrink_workspace_bytes", "lora_backward_workspace_bytes",
    "lora_segments_sched_elems", "lora_base_product_workspace_bytes", "lora_backward_quant_workspace_bytes",
    "MxRows", "MxWeight", "ExpertSegments", "lora_quant_rows_mx", "lora_dequant_rows_mx", "lora_quant_weight_mx",
    "lora_base_product_mx", "lora_base_product_mx_workspace_bytes", "lora_expert_segments", "lora_expert_gather",
    "lora_expert_gather_backward", "lora_expert_combine", "lora_expert_combine_backward", "lora_expert_product_mx",
]

_DTYPES = {torch.bfloat16: LORA_BF16, torch.float32: LORA_F32}


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError(f"element type must be bfloat16 or float32, got {t.dtype}")
    return _DTYPES[t.dtype]


# The current stream's raw handle, without building a torch Stream object per
# call (that costs about as much as the rest of a call's marshalling); the
# public query where this PyTorch build lacks the raw one.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev: torch.device) -> int:
    if _raw_stream is not None:
        return _raw_stream(dev.index if dev.index is not None else torch.cuda.current_device())
    return torch.cuda.current_stream(dev).cuda_stream


def _on_gpu(*ts: Optional[torch.Tensor]) -> None:
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must be on the GPU")


def _fits(name: str, *sizes: int) -> None:
    """ValueError for a size that the C calls' int32 would take as another number."""
    if max(sizes) > 2 ** 31 - 1:
        raise ValueError(f"{name}: sizes are at most 2^31 - 1, got {max(sizes)}")


def _rows(t: torch.Tensor, name: str):
    """(pointer, rows, cols, pitch) of a 2-D tensor whose rows are contiguous."""
    if t.dim() == 2:
        rows, cols = t.shape
        if (rows | cols) >> 31:
            _fits(name, rows, cols)
        pitch, step = t.stride()
        if step == 1:
            # (one row has no pitch: its stride is any number, 1 in a contiguous transpose)
            if rows == 1 and (pitch < cols or pitch % 8):
                pitch = cols
            return t.data_ptr(), rows, cols, pitch
    raise ValueError(f"{name} must be 2-D with contiguous rows")


def _check_batch(name: str, adapters: "AdapterTable", seg: "Segments", T: int, *, x=None, y=None,
                 v=None, r_max: int = 0) -> None:
    """Raise ValueError unless the arguments of one compute call describe one batch.

    The C side sizes its offsets and strides from T, the adapter count, the
    dtype and r_max; arguments from different batches would make the kernels
    index outside the buffers, so they are rejected here, before any enqueue."""
    if seg.T != T:
        raise ValueError(f"{name}: the segments were built for {seg.T} rows, the call has {T}")
    if seg.num_adapters != len(adapters):
        raise ValueError(f"{name}: the segments were built for {seg.num_adapters} adapters, "
                         f"the table has {len(adapters)}")
    if x is not None:
        if x.dtype != adapters.dtype:
            raise ValueError(f"{name}: x is {x.dtype}, the adapters are {adapters.dtype}")
        if x.shape[1] != adapters.d_in:
            raise ValueError(f"{name}: x has {x.shape[1]} columns, the adapters' d_in is {adapters.d_in}")
        if x.device != adapters.device:
            raise ValueError(f"{name}: x and the adapters are on different devices")
    if y is not None:
        if y.dtype != adapters.dtype:
            raise ValueError(f"{name}: y is {y.dtype}, the adapters are {adapters.dtype}")
        if y.shape[1] != adapters.d_out:
            raise ValueError(f"{name}: y has {y.shape[1]} columns, the adapters' d_out is {adapters.d_out}")
        if y.shape[0] != T:
            raise ValueError(f"{name}: y has {y.shape[0]} rows, the call has {T}")
        if y.device != adapters.device:
            raise ValueError(f"{name}: y and the adapters are on different devices")
    if v is not None:
        if v.dtype != torch.float32:
            raise ValueError(f"{name}: v must be float32")
        if v.dim() != 2 or v.shape[0] != T:
            raise ValueError(f"{name}: v must have one row per row of the call ({T})")
        if v.shape[1] < (r_max + 7) // 8 * 8:
            raise ValueError(f"{name}: v needs at least round_up(r_max, 8) = {(r_max + 7) // 8 * 8} columns")
        if v.device != adapters.device:
            raise ValueError(f"{name}: v and the adapters are on different devices")


def lora_abi_version() -> int:
    return _abi.load().lora_abi_version()


def lora_status_string(status: int) -> str:
    return _abi.status_string(status)


def lora_segments_workspace_bytes(T: int, num_adapters: int) -> int:
    return _abi.load().lora_segments_workspace_bytes(T, num_adapters)


def lora_shrink_workspace_bytes(dtype: torch.dtype, T: int, d_in: int, r_max: int) -> int:
    return _abi.load().lora_shrink_workspace_bytes(_DTYPES[dtype], T, d_in, r_max)


def lora_backward_workspace_bytes(dtype: torch.dtype, T_ft: int, d_in: int, d_out: int, r_max: int) -> int:
    return _abi.load().lora_backward_workspace_bytes(_DTYPES[dtype], T_ft, d_in, d_out, r_max)


def lora_segments_sched_elems(T: int, num_adapters: int) -> int:
    return _abi.load().lora_segments_sched_elems(T, num_adapters)


class AdapterTable:
    """Device-resident table of adapters (lora_adapter structs).

    A[a]: [r_a, d_in] and B[a]: [d_out, r_a] tensors on the GPU (kept alive
    by this object); scales[a] multiplies adapter a's delta.
    """

    def __init__(self, A: Sequence[torch.Tensor], B: Sequence[torch.Tensor], scales: Sequence[float]):
        if not (len(A) == len(B) == len(scales)) or len(A) == 0:
            raise ValueError("A, B and scales must have the same nonzero length")
        self.A = list(A)
        self.B = list(B)
        self.scales = [float(s) for s in scales]
        self.dtype = self.A[0].dtype
        self.device = self.A[0].device
        _on_gpu(*self.A, *self.B)
        ranks = []
        host = (_abi.LoraAdapter * len(A))()
        for i, (a, b, s) in enumerate(zip(self.A, self.B, self.scales)):
            if a.dtype != self.dtype or b.dtype != self.dtype or not a.is_contiguous() or not b.is_contiguous():
                raise ValueError("adapter weights must share one dtype and be contiguous")
            if a.dim() != 2 or b.dim() != 2 or b.shape[1] != a.shape[0]:
                raise ValueError("A must be [r, d_in] and B [d_out, r]")
            if a.shape[1] != self.A[0].shape[1] or b.shape[0] != self.B[0].shape[0]:
                raise ValueError("every A must have the same d_in and every B the same d_out")
            if a.device != self.device or b.device != self.device:
                raise ValueError("adapter weights must live on one device")
            host[i] = _abi.LoraAdapter(a.data_ptr(), b.data_ptr(), a.shape[0], s)
            ranks.append(int(a.shape[0]))
        self.ranks = ranks
        self.r_max = max(ranks)
        self.d_in = int(self.A[0].shape[1])
        self.d_out = int(self.B[0].shape[0])
        raw = bytes(host)
        self.table = torch.frombuffer(bytearray(raw), dtype=torch.uint8).to(self.device)

    def __len__(self) -> int:
        return len(self.A)

    @property
    def ptr(self) -> int:
        return self.table.data_ptr()


class GradTable:
    """Device-resident table of fp32 gradient targets (lora_adapter_grad structs).

    dA[a]: [r_a, d_in], dB[a]: [d_out, r_a] float32 GPU tensors, or None for
    adapters that are not trained.
    """

    def __init__(self, dA: Sequence[Optional[torch.Tensor]], dB: Sequence[Optional[torch.Tensor]]):
        if len(dA) != len(dB) or len(dA) == 0:
            raise ValueError("dA and dB must have the same nonzero length")
        self.dA = list(dA)
        self.dB = list(dB)
        host = (_abi.LoraAdapterGrad * len(dA))()
        device = None
        for i, (ga, gb) in enumerate(zip(self.dA, self.dB)):
            if (ga is None) != (gb is None):
                raise ValueError("dA and dB must both be given or both be None")
            if ga is None:
                continue
            _on_gpu(ga, gb)
            if ga.dtype != torch.float32 or gb.dtype != torch.float32:
                raise TypeError("gradients are float32")
            if not ga.is_contiguous() or not gb.is_contiguous():
                raise ValueError("gradients must be contiguous")
            device = ga.device
            host[i] = _abi.LoraAdapterGrad(ga.data_ptr(), gb.data_ptr())
        if device is None:
            raise ValueError("at least one adapter needs gradient buffers")
        self.table = torch.frombuffer(bytearray(bytes(host)), dtype=torch.uint8).to(device)

    @property
    def ptr(self) -> int:
        return self.table.data_ptr()


class _Quant:
    """8-bit floating point matrix: value = code * 2^(scale - 127), one scale per block of 128.

    codes: uint8 (or float8_e4m3fn) [rows, ld], scales: uint8 [.., lds], on one GPU with contiguous
    rows; ld a multiple of 128 and lds of 4 (widths rounded up to these).  The codes of columns from the last value's to
    the end of its block of 128 are zeros."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, rows: int, scale_rows: int, cols: int):
        if codes.dtype not in (torch.uint8, torch.float8_e4m3fn) or scales.dtype != torch.uint8:
            raise TypeError("codes must be uint8 or float8_e4m3fn, scales uint8")
        _on_gpu(codes, scales)
        if codes.device != scales.device:
            raise ValueError("codes and scales must live on one device")
        _fits("an 8-bit matrix", rows, cols)
        block = _abi.LORA_QUANT_BLOCK
        for name, t, r, c, unit in (("codes", codes, rows, -(-cols // block) * block, block),
                                    ("scales", scales, scale_rows, -(-cols // (4 * block)) * 4, 4)):
            if t.dim() != 2 or t.stride(1) != 1 or t.shape[0] != r or t.shape[1] < c:
                raise ValueError(f"{name} must be [{r}, >= {c}] with contiguous rows")
            if r > 1 and (t.stride(0) % unit or t.stride(0) < t.shape[1]):
                raise ValueError(f"the row pitch of {name} must be a multiple of {unit}")
        self.codes, self.scales, self.device = codes, scales, codes.device
        # (one row has no pitch: a slice of a wider matrix may stand at any, its own width is what counts)
        self.c = _abi.LoraQuant(codes.data_ptr(), codes.stride(0) if rows > 1 else -(-cols // block) * block,
                                scales.data_ptr(), scales.stride(0) if scale_rows > 1 else -(-cols // (4 * block)) * 4)

    @staticmethod
    def _buffers(rows: int, scale_rows: int, cols: int, device):
        block = _abi.LORA_QUANT_BLOCK
        nb = -(-cols // block)
        u8 = dict(dtype=torch.uint8, device=device)
        return (torch.empty(rows, nb * block, **u8), torch.full((scale_rows, -(-nb // 4) * 4), 127, **u8))


class QuantRows(_Quant):
    """Rows (activations) in 8 bits: codes [T, >= round_up(d, 128)], scales [T, >= round_up(ceil(d / 128), 4)].

    A slice of rows (q[a:b]) is a QuantRows over the same memory."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, d: int):
        T = int(codes.shape[0])
        super().__init__(codes, scales, T, T, d)
        self.T, self.d = T, int(d)

    @classmethod
    def empty(cls, T: int, d: int, device) -> "QuantRows":
        """Buffers for T rows of d values, contents unset (a checkpoint is filled piece by piece)."""
        return cls(*cls._buffers(T, T, d, device), d)

    def __len__(self) -> int:
        return self.T

    def __getitem__(self, rows: slice) -> "QuantRows":
        if not isinstance(rows, slice) or rows.step not in (None, 1):
            raise TypeError("rows are taken as a slice of consecutive rows")
        return QuantRows(self.codes[rows], self.scales[rows], self.d)


class QuantWeight(_Quant):
    """A weight [d_out, d_in] in 8 bits, 128 x 128 values per scale: codes [d_out, >= round_up(d_in, 128)],
    scales [ceil(d_out / 128), >= round_up(ceil(d_in / 128), 4)]."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, d_out: int, d_in: int):
        super().__init__(codes, scales, d_out, -(-d_out // _abi.LORA_QUANT_BLOCK), d_in)
        self.d_out, self.d_in = int(d_out), int(d_in)


class _Mx:
    """Matrix in microscaled 4 bits: value = code * 2^(scale - 127), one scale per row and 32 columns.

    codes: uint8 [rows, >= round_up(cols, 256) / 2], two e2m1 codes a byte (column 2 i in the low four bits),
    scales: uint8 [rows, >= round_up(cols, 256) / 32], on one GPU with contiguous rows; row pitches multiples of
    128 and 8.  Codes past the last column are zeros, scales of blocks without a column 127."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int):
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        _on_gpu(codes, scales)
        if codes.device != scales.device:
            raise ValueError("codes and scales must live on one device")
        _fits("a 4-bit matrix", rows, cols)
        pad = -(-cols // _abi.LORA_MX_PAD) * _abi.LORA_MX_PAD
        for name, t, c, unit in (("codes", codes, pad // 2, _abi.LORA_MX_PAD // 2),
                                 ("scales", scales, pad // _abi.LORA_MX_BLOCK, _abi.LORA_MX_PAD // _abi.LORA_MX_BLOCK)):
            if t.dim() != 2 or t.stride(1) != 1 or t.shape[0] != rows or t.shape[1] < c:
                raise ValueError(f"{name} must be [{rows}, >= {c}] with contiguous rows")
            if rows > 1 and (t.stride(0) % unit or t.stride(0) < t.shape[1]):
                raise ValueError(f"the row pitch of {name} must be a multiple of {unit}")
        self.codes, self.scales, self.device, self.index = codes, scales, codes.device, codes.get_device()
        # (one row has no pitch: a slice of a wider matrix may stand at any, its own width is what counts)
        self.c = _abi.LoraQuant(codes.data_ptr(), codes.stride(0) if rows > 1 else pad // 2,
                                scales.data_ptr(), scales.stride(0) if rows > 1 else pad // _abi.LORA_MX_BLOCK)

    @staticmethod
    def _buffers(rows: int, cols: int, device):
        pad = -(-cols // _abi.LORA_MX_PAD) * _abi.LORA_MX_PAD
        u8 = dict(dtype=torch.uint8, device=device)
        return torch.empty(rows, pad // 2, **u8), torch.empty(rows, pad // _abi.LORA_MX_BLOCK, **u8)


class MxRows(_Mx):
    """Rows [T, d] in microscaled 4 bits.  A slice of rows (q[a:b]) is a MxRows over the same memory."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, d: int):
        self.T, self.d = int(codes.shape[0]), int(d)
        super().__init__(codes, scales, self.T, self.d)

    @classmethod
    def empty(cls, T: int, d: int, device) -> "MxRows":
        """Buffers for T rows of d values, contents unset (filled piece by piece)."""
        return cls(*cls._buffers(T, d, device), d)

    def as_weight(self, experts: Optional[int] = None) -> "MxWeight":
        """These rows as a weight [T, d], or as `experts` weights [T / experts, d], one below the other."""
        if self.T % (experts or 1):
            raise ValueError(f"{self.T} rows are not {experts} weights")
        return MxWeight(self.codes, self.scales, self.T // (experts or 1), self.d, experts)

    def __len__(self) -> int:
        return self.T

    def __getitem__(self, rows: slice) -> "MxRows":
        if not isinstance(rows, slice) or rows.step not in (None, 1):
            raise TypeError("rows are taken as a slice of consecutive rows")
        return MxRows(self.codes[rows], self.scales[rows], self.d)


class MxWeight(_Mx):
    """A weight [d_out, d_in] in microscaled 4 bits, or `experts` of them, one below the other: codes and scales have
    experts * d_out rows."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, d_out: int, d_in: int, experts: Optional[int] = None):
        if experts is not None and experts < 1:
            raise ValueError("experts must be 1 or more")
        super().__init__(codes, scales, d_out * (experts or 1), d_in)
        self.d_out, self.d_in, self.experts = int(d_out), int(d_in), experts

    def rows(self) -> MxRows:
        """The weight's rows, of all experts, e.g. to restore them (lora_dequant_rows_mx)."""
        return MxRows(self.codes, self.scales, self.d_in)


class Segments:
    """Output of lora_segments_build: rows grouped by adapter (device tensors)."""

    def __init__(self, T: int, num_adapters: int, device: torch.device):
        lib = _abi.load()
        _fits("rows grouped by adapter", T, num_adapters)
        self.T = T
        self.num_adapters = num_adapters
        i32 = dict(dtype=torch.int32, device=device)
        self.counts = torch.zeros(num_adapters, **i32)
        self.offsets = torch.zeros(num_adapters + 1, **i32)
        self.perm = torch.zeros(max(T, 1), **i32)
        self.err = torch.zeros(1, **i32)
        self.sched = torch.zeros(max(1, lib.lora_segments_sched_elems(T, num_adapters)), **i32)
        self.ws = torch.empty(max(1, lib.lora_segments_workspace_bytes(T, num_adapters)), dtype=torch.uint8,
                              device=device)
        self._c = _abi.LoraSegments(self.counts.data_ptr(), self.offsets.data_ptr(), self.perm.data_ptr(),
                                    self.err.data_ptr(), self.sched.data_ptr())

    @property
    def c(self) -> _abi.LoraSegments:
        """The C struct of device pointers (the tensors are allocated once, so it is built once)."""
        return self._c


class ExpertSegments(Segments):
    """Output of lora_expert_segments: the tokens' choices grouped by expert (Segments of tokens * k rows), and pos
    [tokens, k], the place of every choice among the sorted rows (-1: of no expert)."""

    def __init__(self, tokens: int, k: int, num_experts: int, device: torch.device):
        # (one buffer, cleared at once, in place of a tensor and a launch each: a batch of its own shape needs its own
        # segments; every part begins at 16 bytes)
        lib = _abi.load()
        T = tokens * k
        _fits("choices of experts", tokens, k, T, num_experts)
        elems = [num_experts, num_experts + 1, max(T, 1), 1, max(1, lib.lora_segments_sched_elems(T, num_experts)), T]
        parts = torch.zeros(sum((n + 3) // 4 * 4 for n in elems), dtype=torch.int32, device=device).split(
            [m for n in elems for m in (n, -n % 4)])
        self.T, self.num_adapters, self.tokens, self.k = T, num_experts, tokens, k
        self.counts, self.offsets, self.perm, self.err, self.sched = parts[:10:2]
        self.pos = parts[10].view(tokens, k).fill_(-1)
        self.ws = torch.empty(max(1, lib.lora_segments_workspace_bytes(T, num_experts)), dtype=torch.uint8, device=device)
        self.device, self.index = self.pos.device, self.pos.get_device()
        self._c = _abi.LoraSegments(self.counts.data_ptr(), self.offsets.data_ptr(), self.perm.data_ptr(),
                                    self.err.data_ptr(), self.sched.data_ptr())


def lora_segments_build(adapter_ids: torch.Tensor, num_adapters: int, out: Optional[Segments] = None) -> Segments:
    """Group rows by adapter id (-1 = no adapter).  Returns (or refills) a Segments."""
    _on_gpu(adapter_ids)
    if adapter_ids.dtype != torch.int32 or adapter_ids.dim() != 1 or not adapter_ids.is_contiguous():
        raise ValueError("adapter_ids must be a contiguous 1-D int32 tensor")
    T = int(adapter_ids.shape[0])
    seg = out if out is not None else Segments(T, num_adapters, adapter_ids.device)
    if seg.T != T or seg.num_adapters != num_adapters:
        raise ValueError("Segments buffers were sized for another batch")
    st = _abi.load().lora_segments_build(adapter_ids.data_ptr(), T, num_adapters, seg.c, seg.ws.data_ptr(),
                                         seg.ws.numel(), _stream(adapter_ids.device))
    _abi.check("lora_segments_build", st)
    return seg


def lora_segments_build_batch(jobs, num_adapters: int) -> list:
    """Several lora_segments_build calls in one enqueue: jobs = [(adapter_ids, out Segments or None), ...]
    on one device; the one-workgroup builds share launches.  Returns the Segments, in order."""
    segs, raw = [], []
    for ids, out in jobs:
        _on_gpu(ids)
        if ids.dtype != torch.int32 or ids.dim() != 1 or not ids.is_contiguous():
            raise ValueError("adapter_ids must be a contiguous 1-D int32 tensor")
        T = int(ids.shape[0])
        seg = out if out is not None else Segments(T, num_adapters, ids.device)
        if seg.T != T or seg.num_adapters != num_adapters:
            raise ValueError("Segments buffers were sized for another batch")
        segs.append(seg)
        raw.append(_abi.LoraSegmentsJob(ids.data_ptr(), T, seg.c, seg.ws.data_ptr(), seg.ws.numel()))
    if not segs:
        return segs
    arr = (_abi.LoraSegmentsJob * len(raw))(*raw)
    st = _abi.load().lora_segments_build_batch(ctypes.addressof(arr), len(raw), num_adapters,
                                               _stream(jobs[0][0].device))
    _abi.check("lora_segments_build_batch", st)
    return segs


def lora_shrink(x: torch.Tensor, adapters: AdapterTable, seg: Segments, v: Optional[torch.Tensor] = None,
                r_max: Optional[int] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """v[t, :r_a] = A_a x_t (fp32) for every row with an adapter; returns v [T, r_max]."""
    _on_gpu(x)
    px, T, d_in, ldx = _rows(x, "x")
    r_max = adapters.r_max if r_max is None else r_max
    if v is None:
        v = torch.zeros((T, (r_max + 7) // 8 * 8), dtype=torch.float32, device=x.device)
    pv, _, _, ldv = _rows(v, "v")
    _check_batch("lora_shrink", adapters, seg, T, x=x, v=v, r_max=r_max)
    lib = _abi.load()
    if ws is None:  # a caller's workspace is size-checked by the library (LORA_ERR_WORKSPACE)
        ws = torch.empty(max(lib.lora_shrink_workspace_bytes(_dtype_code(x), T, d_in, r_max), 1),
                         dtype=torch.uint8, device=x.device)
    st = lib.lora_shrink(_dtype_code(x), px, ldx, T, d_in, adapters.ptr, len(adapters), r_max, seg.c,
                         pv, ldv, ws.data_ptr(), ws.numel(), _stream(x.device))
    _abi.check("lora_shrink", st)
    return v


def lora_shrink_noalloc(x: torch.Tensor, adapters: AdapterTable, seg: Segments, v: torch.Tensor,
                        r_max: Optional[int] = None) -> torch.Tensor:
    """lora_shrink into the caller's v with the library's static device scratch as its
    workspace: neither the library nor this binding allocates anything.  Calls that
    overlap on one GPU share that scratch and must be ordered by the caller."""
    _on_gpu(x, v)
    px, T, d_in, ldx = _rows(x, "x")
    r_max = adapters.r_max if r_max is None else r_max
    pv, _, _, ldv = _rows(v, "v")
    _check_batch("lora_shrink_noalloc", adapters, seg, T, x=x, v=v, r_max=r_max)
    st = _abi.load().lora_shrink_noalloc(_dtype_code(x), px, ldx, T, d_in, adapters.ptr, len(adapters), r_max, seg.c,
                                         pv, ldv, _stream(x.device))
    _abi.check("lora_shrink_noalloc", st)
    return v


def lora_expand_add(v: torch.Tensor, adapters: AdapterTable, seg: Segments, y: torch.Tensor,
                    r_max: Optional[int] = None) -> torch.Tensor:
    """y[t] += s_a B_a v[t, :r_a] in place; returns y."""
    _on_gpu(v, y)
    pv, T, _, ldv = _rows(v, "v")
    py, Ty, d_out, ldy = _rows(y, "y")
    if Ty != T:
        raise ValueError("v and y must have the same number of rows")
    r_max = adapters.r_max if r_max is None else r_max
    _check_batch("lora_expand_add", adapters, seg, T, y=y, v=v, r_max=r_max)
    st = _abi.load().lora_expand_add(_dtype_code(y), pv, ldv, T, d_out, adapters.ptr, len(adapters), r_max,
                                     seg.c, py, ldy, _stream(y.device))
    _abi.check("lora_expand_add", st)
    return y


def lora_forward(x: torch.Tensor, adapters: AdapterTable, seg: Segments, y: torch.Tensor,
                 v: Optional[torch.Tensor] = None, r_max: Optional[int] = None) -> torch.Tensor:
    """y[t] += s_a B_a A_a x[t] without a workspace; v, if given, receives A_a x[t].

    The library picks the kernels: one launch on rank-16 decode batches; with v
    given on other decode batches or at r_max <= 16, the split calls' kernels
    (bit-equal to lora_shrink + lora_expand_add); otherwise one 64-row-tile launch.
    """
    _on_gpu(x, y, v)
    px, T, d_in, ldx = _rows(x, "x")
    py, Ty, d_out, ldy = _rows(y, "y")
    if Ty != T:
        raise ValueError("x and y must have the same number of rows")
    if y.dtype != x.dtype:
        raise ValueError("x and y must have the same element type")
    pv, ldv = 0, 0
    if v is not None:
        pv, Tv, _, ldv = _rows(v, "v")
        if Tv != T or v.dtype != torch.float32:
            raise ValueError("v must be fp32 with one row per row of x")
    r_max = adapters.r_max if r_max is None else r_max
    _check_batch("lora_forward", adapters, seg, T, x=x, y=y, v=v, r_max=r_max)
    st = _abi.load().lora_forward(_dtype_code(x), px, ldx, T, d_in, d_out, adapters.ptr, len(adapters), r_max,
                                  seg.c, py, ldy, pv or None, ldv, _stream(x.device))
    _abi.check("lora_forward", st)
    return y


def lora_forward_multi(x: torch.Tensor, slices, seg: Segments, r_max: Optional[int] = None) -> None:
    """Several projections of the same x: slices = [(adapters, y[, v]), ...] (1..3 entries).

    For every slice, y[t] += s_a B_a A_a x[t] with that slice's adapter table (same adapter ids),
    bit-equal to lora_forward of that slice alone with the same arguments; the slices that
    lora_forward would run in one launch share one launch (x read once per tile).
    """
    entries = [tuple(e) + (None,) * (3 - len(e)) for e in slices]
    if not 1 <= len(entries) <= _abi.LORA_MAX_SLICES:
        raise ValueError(f"1 to {_abi.LORA_MAX_SLICES} slices")
    _on_gpu(x)
    px, T, d_in, ldx = _rows(x, "x")
    arr = (_abi.LoraSlice * len(entries))()
    n_adapters = len(entries[0][0])
    for i, (table, y, v) in enumerate(entries):
        _on_gpu(y, v)
        py, Ty, d_out, ldy = _rows(y, "y")
        if Ty != T or y.dtype != x.dtype:
            raise ValueError("every y must have x's rows and element type")
        if len(table) != n_adapters:
            raise ValueError("every slice's adapter table must have the same number of entries")
        pv, ldv = 0, 0
        if v is not None:
            pv, Tv, _, ldv = _rows(v, "v")
            if Tv != T or v.dtype != torch.float32:
                raise ValueError("v must be fp32 with one row per row of x")
        arr[i] = _abi.LoraSlice(table.ptr, py, ldy, pv or None, ldv, d_out, 0)
    if r_max is None:
        r_max = max(e[0].r_max for e in entries)
    for table, y, v in entries:
        _check_batch("lora_forward_multi", table, seg, T, x=x, y=y, v=v, r_max=r_max)
    st = _abi.load().lora_forward_multi(_dtype_code(x), px, ldx, T, d_in, arr, len(entries), n_adapters, r_max,
                                        seg.c, _stream(x.device))
    _abi.check("lora_forward_multi", st)


def lora_backward(x: torch.Tensor, dy: torch.Tensor, adapters: AdapterTable, grads: GradTable, seg_ft: Segments,
                  dx: Optional[torch.Tensor] = None, v_saved: Optional[torch.Tensor] = None,
                  r_max: Optional[int] = None, ws: Optional[torch.Tensor] = None) -> None:
    """Accumulate dX (if given), dA and dB of the fine-tuning rows x / dy."""
    _backward("lora_backward", x, dy, adapters, grads, seg_ft, dx, v_saved, r_max, ws, ())


def lora_backward_preemptible(x: torch.Tensor, dy: torch.Tensor, adapters: AdapterTable, grads: GradTable,
                              seg_ft: Segments, grant: torch.Tensor, status: torch.Tensor,
                              dx: Optional[torch.Tensor] = None, v_saved: Optional[torch.Tensor] = None,
                              r_max: Optional[int] = None, ws: Optional[torch.Tensor] = None) -> None:
    """lora_backward that yields while grant[0] == 0; status[0] becomes 0 (ran) or 1 (yielded, outputs untouched).

    grant: int32 tensor on the GPU, or in pinned host memory (``pin_memory=True``), which the
    host may change while the call is queued: the device reads it when the call's gates run."""
    if not status.is_cuda or status.dtype != torch.int32 or status.numel() < 1:
        raise ValueError("status must be an int32 tensor on the GPU")
    if grant.dtype != torch.int32 or grant.numel() < 1:
        raise ValueError("grant must be an int32 tensor")
    if grant.is_cuda:
        grant_ptr = grant.data_ptr()
    elif grant.is_pinned():
        grant_ptr = _abi.host_device_pointer(grant.data_ptr())
    else:
        raise ValueError("grant must be on the GPU or in pinned host memory")
    _backward("lora_backward_preemptible", x, dy, adapters, grads, seg_ft, dx, v_saved, r_max, ws,
              (grant_ptr, status.data_ptr()))


def lora_backward_quant(x: QuantRows, dy: torch.Tensor, adapters: AdapterTable, grads: GradTable, seg_ft: Segments,
                        dx: Optional[torch.Tensor] = None, v_saved: Optional[torch.Tensor] = None,
                        r_max: Optional[int] = None, ws: Optional[torch.Tensor] = None) -> None:
    """lora_backward from the fine-tuning rows' saved 8-bit layer input, read as it is.

    The gradients (+=) are those of lora_backward on lora_dequant_rows(x): dX bit for bit, dA and dB
    with g and v in full."""
    _backward("lora_backward_quant", x, dy, adapters, grads, seg_ft, dx, v_saved, r_max, ws, ())


def _backward(fn, x, dy, adapters, grads, seg_ft, dx, v_saved, r_max, ws, extra) -> None:
    quant = fn == "lora_backward_quant"
    if isinstance(x, QuantRows) != quant:
        raise TypeError("x must be a QuantRows (lora_quant_rows)" if quant else
                        f"{fn}: x must be a tensor (lora_backward_quant takes 8-bit rows)")
    if quant:
        T, d_in, rows = x.T, x.d, (x.c,)
        if x.device != adapters.device:
            raise ValueError(f"{fn}: x and the adapters are on different devices")
        if d_in != adapters.d_in:
            raise ValueError(f"{fn}: x has {d_in} columns, the adapters' d_in is {adapters.d_in}")
    else:
        _on_gpu(x)
        px, T, d_in, ldx = _rows(x, "x")
        rows = (px, ldx)
    _on_gpu(dy, dx, v_saved)
    pdy, Td, d_out, lddy = _rows(dy, "dy")
    if Td != T:
        raise ValueError("x and dy must have the same number of rows")
    pdx, lddx = 0, 0
    if dx is not None:
        pdx, Tx, _, lddx = _rows(dx, "dx")
        if Tx != T or dx.dtype != (adapters.dtype if quant else x.dtype):
            raise ValueError("dx must match x")
        if quant and (dx.shape[1] != d_in or dx.device != adapters.device):
            raise ValueError(f"{fn}: dx must have {d_in} columns on the adapters' device")
    pvs, ldv = 0, 0
    if v_saved is not None:
        pvs, _, _, ldv = _rows(v_saved, "v_saved")
    if len(grads.dA) != len(adapters):
        raise ValueError("the gradient table must have one entry per adapter")
    r_max = adapters.r_max if r_max is None else r_max
    _check_batch(fn, adapters, seg_ft, T, x=None if quant else x, v=v_saved, r_max=r_max)
    if dy.dtype != adapters.dtype or dy.shape[1] != adapters.d_out or dy.device != adapters.device:
        raise ValueError(f"{fn}: dy must be {adapters.dtype} with d_out = {adapters.d_out} columns on the adapters' device")
    for i, (ga, gb) in enumerate(zip(grads.dA, grads.dB)):
        if ga is None:
            continue
        if ga.shape != adapters.A[i].shape or gb.shape != adapters.B[i].shape:
            raise ValueError(f"{fn}: gradient entry {i} must have the shapes of A[{i}] and B[{i}]")
        if ga.device != adapters.device or gb.device != adapters.device:
            raise ValueError(f"{fn}: gradient entry {i} is on another device")
    lib = _abi.load()
    code = _dtype_code(dy if quant else x)
    if ws is None:  # a caller's workspace is size-checked by the library (LORA_ERR_WORKSPACE)
        query = lib.lora_backward_quant_workspace_bytes if quant else lib.lora_backward_workspace_bytes
        ws = torch.empty(max(query(code, T, d_in, d_out, r_max), 1), dtype=torch.uint8, device=x.device)
    st = _launch(x.device, getattr(lib, fn), code, *rows, pdy, lddy, pdx or None, lddx, T, d_in, d_out, adapters.ptr,
                 grads.ptr, len(adapters), r_max, seg_ft.c, pvs or None, ldv, ws.data_ptr(), ws.numel(), *extra)
    _abi.check(fn, st)


_device_index = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(dev: torch.device, fn, *args) -> int:
    """fn(*args, stream) on dev's current stream, with dev the current device (kernels are launched there)."""
    if dev.index is None or dev.index == _device_index():
        return fn(*args, _stream(dev))
    with torch.cuda.device(dev):
        return fn(*args, _stream(dev))


def lora_quant_rows(x: torch.Tensor, out: Optional[QuantRows] = None) -> QuantRows:
    """Save rows x [T, d] (bfloat16 or float32) in 8 bits; out: buffers to fill (QuantRows.empty, or a slice)."""
    _on_gpu(x)
    code, dev = _dtype_code(x), x.device
    px, T, d, ldx = _rows(x, "x")
    if out is None:
        out = QuantRows.empty(T, d, dev)
    elif not isinstance(out, QuantRows):
        raise TypeError("out must be a QuantRows")
    elif out.T != T or out.d != d or out.device != dev:
        raise ValueError(f"out must hold {T} rows of {d} values on x's device")
    _abi.check("lora_quant_rows", _launch(dev, _abi.load().lora_quant_rows, code, px, ldx, T, d, out.c))
    return out


def lora_dequant_rows(q: QuantRows, dtype: torch.dtype = torch.bfloat16,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The rows that q holds, as a tensor [T, d] of dtype (or into out, whose type counts)."""
    if not isinstance(q, QuantRows):
        raise TypeError("q must be a QuantRows")
    if out is None:
        out = torch.empty(q.T, q.d, dtype=dtype, device=q.device)
    _on_gpu(out)
    code = _dtype_code(out)
    px, T, d, ldx = _rows(out, "out")
    dev = q.device
    if T != q.T or d != q.d or out.device != dev:
        raise ValueError(f"out must be [{q.T}, {q.d}] on q's device")
    _abi.check("lora_dequant_rows", _launch(dev, _abi.load().lora_dequant_rows, code, q.c, T, d, px, ldx))
    return out


def lora_quant_weight(w: torch.Tensor, transpose: bool = False, out: Optional[QuantWeight] = None) -> QuantWeight:
    """A frozen weight [d_out, d_in] (bfloat16 or float32) in 8 bits; transpose: the form of its transpose."""
    _on_gpu(w)
    code = _dtype_code(w)
    pw, d_out, d_in, ldw = _rows(w, "w")
    rows, cols = (d_in, d_out) if transpose else (d_out, d_in)
    if out is None:
        out = QuantWeight(*QuantWeight._buffers(rows, -(-rows // _abi.LORA_QUANT_BLOCK), cols, w.device), rows, cols)
    elif not isinstance(out, QuantWeight):
        raise TypeError("out must be a QuantWeight")
    elif out.d_out != rows or out.d_in != cols or out.device != w.device:
        raise ValueError(f"out must be a [{rows}, {cols}] weight on w's device")
    st = _launch(w.device, _abi.load().lora_quant_weight, code, pw, ldw, d_out, d_in, int(bool(transpose)), out.c)
    _abi.check("lora_quant_weight", st)
    return out


def lora_base_product_workspace_bytes(T: int, d_in: int, d_out: int) -> int:
    """Not monotone in T; never more than LORA_BASE_PRODUCT_MAX_WORKSPACE (128 MiB)."""
    return _abi.load().lora_base_product_workspace_bytes(T, d_in, d_out)


def lora_base_product(x: QuantRows, w: QuantWeight, y: Optional[torch.Tensor] = None, accumulate: bool = False,
                      dtype: torch.dtype = torch.bfloat16, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = W x for every row (accumulate: y += W x); without y, a new tensor [T, d_out] of dtype.

    Sums are fp32, rounded once.  float32 y sums exact products; for bfloat16 y the matrix instruction cuts
    each of the 8 products of columns 8 i .. 8 i + 7 at 2^-13 of the largest (lora_batch.h states the bound):
    a hundredth of y's rounding on ordinary rows, more only where large products of different columns cancel."""
    if not isinstance(x, QuantRows) or not isinstance(w, QuantWeight):
        raise TypeError("x must be a QuantRows and w a QuantWeight")
    if x.d != w.d_in or x.device != w.device:
        raise ValueError(f"x has {x.d} columns on {x.device}, w has d_in = {w.d_in} on {w.device}")
    dev = x.device
    if y is None:
        if accumulate:
            raise ValueError("accumulate needs y")
        y = torch.empty(x.T, w.d_out, dtype=dtype, device=dev)
    _on_gpu(y)
    code = _dtype_code(y)
    py, T, d_out, ldy = _rows(y, "y")
    if T != x.T or d_out != w.d_out or y.device != dev:
        raise ValueError(f"y must be [{x.T}, {w.d_out}] on x's device")
    lib = _abi.load()
    if ws is None:  # a caller's workspace is size-checked by the library (LORA_ERR_WORKSPACE)
        ws = torch.empty(max(lib.lora_base_product_workspace_bytes(T, x.d, d_out), 1), dtype=torch.uint8, device=dev)
    elif ws.device != dev or not ws.is_contiguous():
        raise ValueError("ws must be contiguous on x's device")
    st = _launch(dev, lib.lora_base_product, code, x.c, T, x.d, w.c, d_out, py, ldy, 1 if accumulate else 0,
                 ws.data_ptr(), ws.nbytes)
    _abi.check("lora_base_product", st)
    return y


def lora_backward_quant_workspace_bytes(dtype: torch.dtype, T_ft: int, d_in: int, d_out: int, r_max: int) -> int:
    return _abi.load().lora_backward_quant_workspace_bytes(_DTYPES[dtype], T_ft, d_in, d_out, r_max)


def _launch_on(index: int, fn, *args) -> int:
    """fn(*args, stream) on the current stream of the device with that index, made the current device."""
    if index == _device_index() and _raw_stream is not None:
        return fn(*args, _raw_stream(index))
    return _launch(torch.device("cuda", index), fn, *args)


def _matrix(fn: str, t: torch.Tensor, name: str, rows: int, index: int):
    """(pointer, columns, pitch, type code) of a 2-D tensor of `rows` rows, contiguous each, on the device with that index."""
    shape, stride = t.shape, t.stride()
    code = _DTYPES.get(t.dtype)
    if len(shape) == 2 and stride[1] == 1 and shape[0] == rows and t.get_device() == index and code is not None:
        if (shape[0] | shape[1]) >> 31:
            _fits(f"{fn}: {name}", *shape)
        # (one row has no pitch: its stride is any number, 1 in a contiguous transpose)
        return t.data_ptr(), shape[1], stride[0] if rows > 1 else shape[1], code
    _on_gpu(t)
    _dtype_code(t)
    _rows(t, name)
    raise ValueError(f"{fn}: {name} must have {rows} rows on cuda:{index}, it has {shape[0]} on {t.device}")


def lora_quant_rows_mx(x: torch.Tensor, out: Optional[MxRows] = None) -> MxRows:
    """Save rows x [T, d] (bfloat16 or float32) in microscaled 4 bits; out: buffers to fill (MxRows.empty, or a slice)."""
    if out is None:
        _on_gpu(x)
        _dtype_code(x)
        _, T, d, _ = _rows(x, "x")
        out = MxRows.empty(T, d, x.device)
    elif not isinstance(out, MxRows):
        raise TypeError("out must be a MxRows")
    px, d, ldx, code = _matrix("lora_quant_rows_mx", x, "x", out.T, out.index)
    if d != out.d:
        raise ValueError(f"out must hold rows of {d} values")
    st = _launch_on(out.index, _abi.load().lora_quant_rows_mx, code, px, ldx, out.T, d, out.c)
    if st:
        _abi.check("lora_quant_rows_mx", st)
    return out


def lora_dequant_rows_mx(q, dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of q (MxRows, or a MxWeight's rows), as a tensor of dtype (or into out, whose type counts)."""
    if isinstance(q, MxRows):
        T, d = q.T, q.d
    elif isinstance(q, MxWeight):
        T, d = q.d_out * (q.experts or 1), q.d_in
    else:
        raise TypeError("q must be a MxRows or a MxWeight")
    if out is None:
        out = torch.empty(T, d, dtype=dtype, device=q.device)
    px, cols, ldx, code = _matrix("lora_dequant_rows_mx", out, "out", T, q.index)
    if cols != d:
        raise ValueError(f"out must be [{T}, {d}]")
    st = _launch_on(q.index, _abi.load().lora_dequant_rows_mx, code, q.c, T, d, px, ldx)
    if st:
        _abi.check("lora_dequant_rows_mx", st)
    return out


def lora_quant_weight_mx(w: torch.Tensor, transpose: bool = False, out: Optional[MxWeight] = None) -> MxWeight:
    """A frozen weight [d_out, d_in], or the weights [experts, d_out, d_in], in microscaled 4 bits with a scale for
    32 x 32 values; transpose: the form of the transpose, with the same values."""
    _on_gpu(w)
    code, dev = _dtype_code(w), w.device
    experts = w.shape[0] if w.dim() == 3 else None
    parts = w.unbind(0) if experts is not None else (w,)
    if not parts:
        raise ValueError("w holds no weight")
    _, d_out, d_in, _ = _rows(parts[0], "w")
    rows, cols = (d_in, d_out) if transpose else (d_out, d_in)
    if out is None:
        out = MxWeight(*MxWeight._buffers(rows * len(parts), cols, dev), rows, cols, experts)
    elif not isinstance(out, MxWeight):
        raise TypeError("out must be a MxWeight")
    elif out.d_out != rows or out.d_in != cols or (out.experts or 1) != len(parts) or out.device != dev:
        raise ValueError(f"out must hold {len(parts)} [{rows}, {cols}] weights on w's device")
    lib = _abi.load()
    q = out.c
    for e, part in enumerate(parts):
        pw, _, _, ldw = _rows(part, "w")
        c = _abi.LoraQuant(q.codes + e * rows * q.ld, q.ld, q.scales + e * rows * q.lds, q.lds)
        st = _launch(dev, lib.lora_quant_weight_mx, code, pw, ldw, d_out, d_in, int(bool(transpose)), c)
        _abi.check("lora_quant_weight_mx", st)
    return out


def lora_base_product_mx_workspace_bytes(T: int, d_in: int, d_out: int) -> int:
    """Not monotone in T; never more than LORA_BASE_PRODUCT_MAX_WORKSPACE (128 MiB)."""
    return _abi.load().lora_base_product_mx_workspace_bytes(T, d_in, d_out)


def _mx_operands(fn: str, x, w, y, accumulate: bool, dtype, cut: bool, new):
    """Checked (x_bits, y, its pointer, pitch and type code) of a product of rows x (MxRows or QuantRows) and a 4-bit weight w."""
    bits = 4 if isinstance(x, MxRows) else 8 if isinstance(x, QuantRows) else 0
    if not bits or not isinstance(w, MxWeight):
        raise TypeError(f"{fn}: x must be a MxRows or a QuantRows and w a MxWeight")
    if x.d != w.d_in or x.codes.get_device() != w.index:
        raise ValueError(f"{fn}: x has {x.d} columns on {x.device}, w has d_in = {w.d_in} on {w.device}")
    if y is None:
        if accumulate:
            raise ValueError(f"{fn}: accumulate needs y")
        y = new(x.T, w.d_out, dtype=dtype, device=x.device)
    py, d_out, ldy, code = _matrix(fn, y, "y", x.T, w.index)
    if d_out != w.d_out:
        raise ValueError(f"{fn}: y must be [{x.T}, {w.d_out}]")
    if cut:
        if bits != 8 or code != LORA_BF16:
            raise ValueError(f"{fn}: products are cut of 8-bit rows with bfloat16 y alone")
        bits |= _abi.LORA_MX_CUT
    return bits, y, py, ldy, code


def lora_base_product_mx(x, w: MxWeight, y: Optional[torch.Tensor] = None, accumulate: bool = False,
                         dtype: torch.dtype = torch.bfloat16, ws: Optional[torch.Tensor] = None,
                         cut: bool = False) -> torch.Tensor:
    """y = W x for every row (accumulate: y += W x) with a 4-bit weight; x: MxRows (4 bits) or QuantRows (8 bits);
    without y, a new tensor [T, d_out] of dtype.

    Sums are fp32 of exact products, rounded once.  cut, for 8-bit rows with bfloat16 y: the matrix instruction may cut
    the products, as in lora_base_product, for half of the work of a large product."""
    fn = "lora_base_product_mx"
    bits, y, py, ldy, code = _mx_operands(fn, x, w, y, accumulate, dtype, cut, torch.empty)
    if w.experts is not None:
        raise ValueError(f"{fn}: w holds several experts' weights (lora_expert_product_mx)")
    lib = _abi.load()
    if ws is None:  # a caller's workspace is size-checked by the library (LORA_ERR_WORKSPACE)
        ws = torch.empty(max(lib.lora_base_product_mx_workspace_bytes(x.T, x.d, w.d_out), 1), dtype=torch.uint8, device=x.device)
    elif ws.get_device() != w.index or not ws.is_contiguous():
        raise ValueError(f"{fn}: ws must be contiguous on x's device")
    st = _launch_on(w.index, lib.lora_base_product_mx, code, bits, x.c, x.T, x.d, w.c, w.d_out, py, ldy, 1 if accumulate else 0,
                    ws.data_ptr(), ws.nbytes)
    if st:
        _abi.check(fn, st)
    return y


def lora_expert_segments(expert_ids: torch.Tensor, num_experts: int, out: Optional[ExpertSegments] = None) -> ExpertSegments:
    """Group the choices expert_ids [tokens, k] (int32, -1 = none) by expert.  Returns (or refills) an ExpertSegments."""
    _on_gpu(expert_ids)
    if expert_ids.dtype != torch.int32 or expert_ids.dim() != 2 or not expert_ids.is_contiguous():
        raise ValueError("expert_ids must be a contiguous 2-D int32 tensor")
    T, k = expert_ids.shape
    index = expert_ids.get_device()
    seg = out if out is not None else ExpertSegments(T, k, num_experts, expert_ids.device)
    if not isinstance(seg, ExpertSegments):
        raise TypeError("out must be an ExpertSegments")
    if seg.tokens != T or seg.k != k or seg.num_adapters != num_experts or seg.index != index:
        raise ValueError("ExpertSegments buffers were sized for another batch")
    st = _launch_on(index, _abi.load().lora_expert_segments, expert_ids.data_ptr(), T, k, num_experts, seg.c, seg.pos.data_ptr(),
                    seg.ws.data_ptr(), seg.ws.nbytes)
    if st:
        _abi.check("lora_expert_segments", st)
    return seg


def _expert_segments(fn: str, seg) -> None:
    if not isinstance(seg, ExpertSegments):
        raise TypeError(f"{fn}: seg must be an ExpertSegments (lora_expert_segments)")
    if seg.index < 0:
        raise ValueError("tensors must be on the GPU")


def _same(fn: str, name: str, d: int, code: int, d0: int, code0: int, p: int = 0, p0: int = -1) -> None:
    if d != d0 or code != code0:
        raise ValueError(f"{fn}: {name} must have {d0} columns of the same type")
    if p and p == p0:  # (another token's row would be written before it is read)
        raise ValueError(f"{fn}: {name} is the rows that are read")


def _router_weights(fn: str, seg: ExpertSegments, w: torch.Tensor, name: str = "w") -> int:
    if w.dtype is not torch.float32 or w.shape != seg.pos.shape or not w.is_contiguous() or w.get_device() != seg.index:
        raise ValueError(f"{fn}: {name} must be float32 [{seg.tokens}, {seg.k}], contiguous, on the segments' device")
    return w.data_ptr()


def lora_expert_gather(x: torch.Tensor, seg: ExpertSegments, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[pos[t, j]] = x[t]: every token's row at the places of its choices, sorted by expert.  y [tokens * k, d]: rows
    behind the last expert's are left as they are (zeros in a new y)."""
    fn = "lora_expert_gather"
    _expert_segments(fn, seg)
    px, d, ldx, code = _matrix(fn, x, "x", seg.tokens, seg.index)
    if y is None:
        y = torch.zeros(seg.T, d, dtype=x.dtype, device=x.device)
    py, dy, ldy, cy = _matrix(fn, y, "y", seg.T, seg.index)
    _same(fn, "y", dy, cy, d, code, py, px)
    st = _launch_on(seg.index, _abi.load().lora_expert_gather, code, px, ldx, seg.tokens, d, seg.k, seg.pos.data_ptr(), py, ldy)
    if st:
        _abi.check(fn, st)
    return y


def lora_expert_gather_backward(dy: torch.Tensor, seg: ExpertSegments, dx: Optional[torch.Tensor] = None,
                                accumulate: bool = False) -> torch.Tensor:
    """The gather's gradient: dx[t] = sum_j dy[pos[t, j]] (accumulate: +=), in fp32, rounded once."""
    fn = "lora_expert_gather_backward"
    _expert_segments(fn, seg)
    pdy, d, lddy, code = _matrix(fn, dy, "dy", seg.T, seg.index)
    if dx is None:
        if accumulate:
            raise ValueError(f"{fn}: accumulate needs dx")
        dx = torch.empty(seg.tokens, d, dtype=dy.dtype, device=dy.device)
    pdx, d2, lddx, c2 = _matrix(fn, dx, "dx", seg.tokens, seg.index)
    _same(fn, "dx", d2, c2, d, code, pdx, pdy)
    st = _launch_on(seg.index, _abi.load().lora_expert_gather_backward, code, pdy, lddy, seg.tokens, d, seg.k, seg.pos.data_ptr(),
                    pdx, lddx, 1 if accumulate else 0)
    if st:
        _abi.check(fn, st)
    return dx


def lora_expert_combine(o: torch.Tensor, w: torch.Tensor, seg: ExpertSegments, y: Optional[torch.Tensor] = None,
                        accumulate: bool = False) -> torch.Tensor:
    """y[t] = sum_j w[t, j] o[pos[t, j]] (accumulate: +=), in fp32, rounded once; o [tokens * k, d] sorted by expert,
    w [tokens, k] float32."""
    fn = "lora_expert_combine"
    _expert_segments(fn, seg)
    po, d, ldo, code = _matrix(fn, o, "o", seg.T, seg.index)
    pw = _router_weights(fn, seg, w)
    if y is None:
        if accumulate:
            raise ValueError(f"{fn}: accumulate needs y")
        y = torch.empty(seg.tokens, d, dtype=o.dtype, device=o.device)
    py, dy, ldy, cy = _matrix(fn, y, "y", seg.tokens, seg.index)
    _same(fn, "y", dy, cy, d, code, py, po)
    st = _launch_on(seg.index, _abi.load().lora_expert_combine, code, po, ldo, seg.tokens, d, seg.k, seg.pos.data_ptr(), pw, py, ldy,
                    1 if accumulate else 0)
    if st:
        _abi.check(fn, st)
    return y


def lora_expert_combine_backward(dy: torch.Tensor, o: Optional[torch.Tensor], w: torch.Tensor, seg: ExpertSegments,
                                 d_o: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None, *,
                                 need_d_o: bool = True, need_dw: bool = True):
    """The combine's gradient: d_o[pos[t, j]] = w[t, j] dy[t] and dw[t, j] = <dy[t], o[pos[t, j]]> (float32; 0 for a
    choice of no expert).  Returns (d_o, dw).  Rows of d_o behind the last expert's are left as they are (zeros in a
    new d_o); d_o may be o.  One of them that is not needed is not computed (None); without dw, o is not read and may be
    None."""
    fn = "lora_expert_combine_backward"
    _expert_segments(fn, seg)
    if not need_d_o and not need_dw or (d_o is not None and not need_d_o) or (dw is not None and not need_dw):
        raise ValueError(f"{fn}: one gradient at least is computed, and none that is not needed is passed")
    pdy, d, lddy, code = _matrix(fn, dy, "dy", seg.tokens, seg.index)
    po = ldo = pd = ldd = pdw = 0
    if o is not None:
        po, d1, ldo, c1 = _matrix(fn, o, "o", seg.T, seg.index)
        _same(fn, "o", d1, c1, d, code)
    elif need_dw:
        raise ValueError(f"{fn}: dw needs o")
    pw = _router_weights(fn, seg, w)
    if need_d_o:
        if d_o is None:
            d_o = torch.zeros(seg.T, d, dtype=dy.dtype, device=dy.device)
        pd, d2, ldd, c2 = _matrix(fn, d_o, "d_o", seg.T, seg.index)
        _same(fn, "d_o", d2, c2, d, code, pd, pdy)
    if need_dw:
        if dw is None:
            dw = torch.empty(seg.tokens, seg.k, dtype=torch.float32, device=dy.device)
        pdw = _router_weights(fn, seg, dw, "dw")
    st = _launch_on(seg.index, _abi.load().lora_expert_combine_backward, code, pdy, lddy, po, ldo, seg.tokens, d, seg.k,
                    seg.pos.data_ptr(), pw, pd, ldd, pdw)
    if st:
        _abi.check(fn, st)
    return d_o, dw


def lora_expert_product_mx(x, w: MxWeight, seg: Segments, y: Optional[torch.Tensor] = None, accumulate: bool = False,
                           dtype: torch.dtype = torch.bfloat16, cut: bool = False) -> torch.Tensor:
    """y[i] = W_e x[i] (accumulate: +=) for every sorted row i of expert e, each expert with its own 4-bit weight, in
    one launch.  x: MxRows or QuantRows of the sorted rows; w: MxWeight with experts.  Rows behind the last expert's
    are left as they are (zeros in a new y).  Precision, and cut: as lora_base_product_mx."""
    fn = "lora_expert_product_mx"
    if not isinstance(seg, Segments):
        raise TypeError(f"{fn}: seg must be a Segments (lora_expert_segments)")
    bits, y, py, ldy, code = _mx_operands(fn, x, w, y, accumulate, dtype, cut, torch.zeros)
    experts = w.experts or 1
    if seg.T != x.T or seg.num_adapters != experts or seg.offsets.get_device() != w.index:
        raise ValueError(f"{fn}: the segments are of {seg.T} rows and {seg.num_adapters} experts on {seg.offsets.device}, the call "
                         f"has {x.T} and {experts} on {w.device}")
    st = _launch_on(w.index, _abi.load().lora_expert_product_mx, code, bits, x.c, x.T, x.d, w.c, experts, w.d_out, seg.c, py, ldy,
                    1 if accumulate else 0)
    if st:
        _abi.check(fn, st)
    return y


def lora_adamw_step(tensors, *, step: int, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                    weight_decay: float = 0.01, grad_scale: float = 1.0, zero_grad: bool = False) -> None:
    """One AdamW step over a list of (w, grad, m, v[, master]) tensors (in place, one launch).

    w: bfloat16 or float32 weights (all entries one element type); grad, m, v and the
    optional master copy: float32 with w's element count, contiguous.
    """
    entries = [tuple(e) + (None,) * (5 - len(e)) for e in tensors]
    if len(entries) > _abi.LORA_ADAMW_MAX_TENSORS:
        raise ValueError(f"at most {_abi.LORA_ADAMW_MAX_TENSORS} tensors per step")
    arr = (_abi.LoraAdamwTensor * max(1, len(entries)))()
    dtype = None
    dev = None
    for i, (w, grad, m, v, master) in enumerate(entries):
        _on_gpu(w, grad, m, v, master)
        code = _dtype_code(w)
        if dtype is not None and code != dtype:
            raise ValueError("all weights of one step must share their element type")
        dtype, dev = code, w.device
        for name, t in (("w", w), ("grad", grad), ("m", m), ("v", v), ("master", master)):
            if t is None and name != "master":
                raise ValueError(f"{name} is required")
            if t is not None and (not t.is_contiguous() or t.numel() != w.numel()):
                raise ValueError(f"{name} must be contiguous with w's element count")
            if t is not None and name != "w" and t.dtype != torch.float32:
                raise ValueError(f"{name} must be float32")
        arr[i] = _abi.LoraAdamwTensor(w.data_ptr(), master.data_ptr() if master is not None else None,
                                      grad.data_ptr(), m.data_ptr(), v.data_ptr(), w.numel())
    hp = _abi.LoraAdamwParams(lr, betas[0], betas[1], eps, weight_decay, grad_scale, int(step), int(bool(zero_grad)))
    stream = _stream(dev) if dev is not None else 0
    st = _abi.load().lora_adamw_step(LORA_BF16 if dtype is None else dtype, arr, len(entries), hp, stream or None)
    _abi.check("lora_adamw_step", st)
