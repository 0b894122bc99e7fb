"""Limits of the 8-bit calls and of the calls beside them that hold without a GPU:
workspace sizes, refusals, and which kernels the tests' shapes reach."""
import pytest
import torch

from expand_token_adapter_amd import _abi

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
