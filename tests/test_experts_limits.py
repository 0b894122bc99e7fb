"""The most rows that the experts' calls take, as documented: one more is refused as unsupported.  Nothing is enqueued:
what a call does take is refused for an output that is its input, which is checked behind the size."""
import pytest

from expand_token_adapter_amd import _abi

AT, FAR = 1 << 20, 1 << 50  # addresses that no check reads
BAD, UNS = _abi.LORA_ERR_INVALID_ARG, _abi.LORA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


@pytest.mark.parametrize("d", [8, 16, 24, 512, 4096, 8192])
def test_rows_there_and_back(lib, d):
    most = (2 ** 35 - 2048) // d
    for T in (most, most + 1):
        if T > 2 ** 31 - 1:
            continue
        want = UNS if T > most else BAD
        assert lib.lora_expert_gather(0, AT, d, T, d, 1, FAR, AT, d, None) == want
        assert lib.lora_expert_gather_backward(1, AT, d, T, d, 1, FAR, AT, d, 0, None) == want
        assert lib.lora_expert_combine(0, AT, d, T, d, 1, FAR, FAR, AT, d, 0, None) == want


@pytest.mark.parametrize("d,most", [(8, 2 ** 26 - 4), (512, 2 ** 26 - 4), (2040, 2 ** 26 - 4), (2048, 2 ** 24 - 1), (8192, 2 ** 24 - 1)])
def test_gradients_of_the_combine(lib, d, most):
    for T in (2 ** 24 - 1, 2 ** 24, most, most + 1, 2 ** 31 - 1):
        want = BAD if T <= most else UNS
        # (dy is where d_o shall be)
        assert lib.lora_expert_combine_backward(0, AT, d, None, 0, T, d, 1, FAR, FAR, AT, d, None, None) == want, T


def test_the_combine_and_its_gradient_take_the_same_wide_rows(lib):
    """From 512 columns on, what the combine takes its gradient takes."""
    for d in (512, 1024, 2040, 2048, 4096):
        T = (2 ** 35 - 2048) // d
        assert lib.lora_expert_combine(0, AT, d, T, d, 1, FAR, FAR, AT, d, 0, None) == BAD
        assert lib.lora_expert_combine_backward(0, AT, d, None, 0, T, d, 1, FAR, FAR, AT, d, None, None) == BAD
