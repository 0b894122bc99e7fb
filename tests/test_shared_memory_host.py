"""Arguments of the experts' calls that share memory: found whatever their pitches, and refused by every call before
anything is enqueued.  (Addresses here are never read: each call is refused.)"""
import os
import random
import subprocess

import pytest

from expand_token_adapter_amd import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD = _abi.LORA_ERR_INVALID_ARG
AT = 1 << 20

ASK = """
#include <stdio.h>
#include "host_checks.h"
using namespace lora;
int main() {
    long long v[8];
    while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld", v, v + 1, v + 2, v + 3, v + 4, v + 5, v + 6, v + 7) == 8) {
        const RowSpan a = RowSpan::matrix((void*)v[0], v[1], v[2], v[3], 1), b = RowSpan::matrix((void*)v[4], v[5], v[6], v[7], 1);
        printf("%d%d\\n", shares_memory(a, b), shares_memory(b, a));
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def shares(tmp_path_factory):
    """[(address, rows, bytes of a row, pitch) of two matrices] -> whether they share a byte, asked both ways."""
    d = tmp_path_factory.mktemp("shares")
    (d / "ask.cpp").write_text(ASK)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "expand_token_adapter_amd", "csrc"), str(d / "ask.cpp"), "-o",
                    str(d / "ask")], check=True)

    def ask(pairs):
        text = "".join(" ".join(map(str, a + b)) + "\n" for a, b in pairs)
        out = subprocess.run([str(d / "ask")], input=text, check=True, capture_output=True, text=True).stdout.split()
        assert len(out) == len(pairs) and set(out) <= {"00", "11"}
        return [o == "11" for o in out]

    return ask


def test_every_layout_of_small_matrices(shares):
    rng = random.Random(2)

    def matrix(pitch=None):
        width = rng.randint(1, 6)
        return (1000 + rng.randint(0, 60), rng.randint(1, 7), width, max(width, pitch or rng.randint(width, 14)))

    pairs = []
    for _ in range(60000):
        a = matrix()
        pairs.append((a, matrix(a[3] if rng.random() < 0.5 else None)))
    taken = lambda m: {m[0] + i * m[3] + c for i in range(m[1]) for c in range(m[2])}
    want = [bool(taken(a) & taken(b)) for a, b in pairs]
    assert shares(pairs) == want
    assert 0.2 < sum(want) / len(want) < 0.8


def test_large_matrices_and_pitches(shares):
    big, far = 2 ** 31 - 1, 2 ** 62
    cases = [((AT, big, 16, 32), (AT + 16, big, 16, 32), False), ((AT, big, 16, 32), (AT + 15, big, 16, 32), True),
             ((AT, big, 16, 32), (AT + 16 + 32 * (big - 1), 5, 16, 32), False), ((AT, big, 16, 32), (AT + 32 * (big - 1), 5, 16, 32), True),
             ((AT, 4, 16, far), (AT + 16, 1, far - 16, far), False), ((AT, 4, 16, far), (AT + 16, 1, far - 15, far), True),
             ((AT, 1, 64, 64), (AT + 64, big, 64, 128), False), ((AT + 64, 1, 64, 64), (AT, big, 64, 192), False)]
    assert shares([c[:2] for c in cases]) == [c[2] for c in cases]


# T = 10 tokens, k = 3, d = 64 bf16 columns: rows of 128 bytes, pitch 80 columns = 160 bytes
T, K, D, LD = 10, 3, 64, 80
NX, NY = (T - 1) * LD * 2 + D * 2, (T * K - 1) * LD * 2 + D * 2  # bytes of the tokens' and of the choices' rows


def _refused(fn, *args):
    assert getattr(_abi.load(), fn)(*args) == BAD


@pytest.mark.parametrize("by", [-NX + 16, -160, -96, 0, 64, 160, NY - 128, NY - 16])
def test_rows_that_overlap_are_refused(by):
    far = AT + (1 << 18)
    other = AT + by
    _refused("lora_expert_gather", 0, other, LD, T, D, K, far, AT, LD, None)
    _refused("lora_expert_gather_backward", 0, AT, LD, T, D, K, far, other, LD, 0, None)
    _refused("lora_expert_combine", 0, AT, LD, T, D, K, far, far, other, LD, 1, None)
    _refused("lora_expert_combine_backward", 0, other, LD, far, LD, T, D, K, far + 65536, far + 65536, AT, LD, far + 65536 * 2, None)


def test_rows_in_place_need_the_same_pitch():
    far = AT + (1 << 18)
    for ld in (72, 88, 160):
        _refused("lora_expert_combine_backward", 0, far, LD, AT, LD, T, D, K, far + 65536, far + 65536, AT, ld, far + 65536 * 2, None)
    for by in (16, 160, -320):
        _refused("lora_expert_combine_backward", 0, far, LD, AT, LD, T, D, K, far + 65536, far + 65536, AT + by, LD, far + 65536 * 2, None)


@pytest.mark.parametrize("by", [-112, -4, 0, 4, 116])
def test_choices_that_overlap_outputs_are_refused(by):
    """Places, weights and their gradient: 120 bytes each."""
    a, b, c = AT + (1 << 18), AT + (1 << 19), AT + (1 << 20)
    end = (T * K - 1) * LD * 2 + D * 2
    for at in (AT + max(by, 0), AT + end - 4 if by > 0 else AT + by):
        _refused("lora_expert_gather", 0, a, LD, T, D, K, at, AT, LD, None)
        _refused("lora_expert_combine_backward", 0, a, LD, b, LD, T, D, K, at, c, AT, LD, c + 4096, None)
        _refused("lora_expert_combine_backward", 0, a, LD, b, LD, T, D, K, c, at, AT, LD, c + 4096, None)
        _refused("lora_expert_combine_backward", 0, a, LD, b, LD, T, D, K, c, c, AT, LD, at, None)  # d_o and dw
        _refused("lora_expert_combine_backward", 0, AT, LD, b, LD, T, D, K, c, c, None, 0, AT + max(by, 0), None)  # dw over dy
        _refused("lora_expert_combine_backward", 0, b, LD, AT, LD, T, D, K, c, c, None, 0, AT + max(by, 0), None)  # dw over o
    _refused("lora_expert_gather_backward", 0, a, LD, T, D, K, AT + max(by, 0), AT, LD, 0, None)
    _refused("lora_expert_combine", 0, a, LD, T, D, K, AT + max(by, 0), c, AT, LD, 0, None)
    _refused("lora_expert_combine", 0, a, LD, T, D, K, c, AT + max(by, 0), AT, LD, 0, None)
    _refused("lora_expert_combine_backward", 0, a, LD, b, LD, T, D, K, c + 4096, c, None, 0, c + by, None)  # dw over w
    _refused("lora_expert_combine_backward", 0, a, LD, b, LD, T, D, K, c + by, AT, None, 0, c, None)  # dw over the places
    seg = _abi.LoraSegments(a, a, a, a, a)
    _refused("lora_expert_segments", AT, T, K, 4, seg, AT + by, b, 1 << 20, None)


@pytest.mark.parametrize("bits", [4, 8])
def test_products_over_their_operands_are_refused(bits):
    far = AT + (1 << 22)
    q = lambda at, ld=None: _abi.LoraQuant(at, ld or (128 if bits == 4 else 256), far + 65536, 8)
    w = lambda at, s=far + 131072: _abi.LoraQuant(at, 128, s, 8)
    seg = lambda at=far + 262144: _abi.LoraSegments(at, at, at, at, at)
    call = lambda x, w, s: _refused("lora_expert_product_mx", 0, bits, x, 30, 200, w, 3, 64, s, AT, 64, 0, None)
    call(q(AT + 128), w(far), seg())
    call(q(far), w(AT - 128), seg())
    call(q(far), w(AT - (3 * 64 - 1) * 128), seg())
    call(q(far), w(far, AT + 128 * 29), seg())
    call(q(far), w(far), seg(AT + 30 * 128 - 16))
    call(_abi.LoraQuant(far, 256, AT + 64, 8), w(far), seg())
