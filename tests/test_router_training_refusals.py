"""Calls of the gradient norm and clipping that have no right answer, refused on
the host (no call here reaches a launch)."""
import os
import struct

import pytest

from mixture_experts_layer_15_amd import binding as B

BASE = 0x10000  # never dereferenced
BAD = B.MOE_ERR_INVALID_ARGUMENT


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from mixture_experts_layer_15_amd import build
        build.build()
    return B.load_library()


def pack(*rows):
    return struct.pack(B._GRAD * len(rows), *[v for r in rows for v in r])


@pytest.mark.parametrize("dtype,size", [(B.MOE_F32, 4), (B.MOE_BF16, 2)])
@pytest.mark.parametrize("word", [0, 25, 49])
def test_the_norm_may_not_lie_in_what_clipping_writes(lib, dtype, size, word):
    """Workgroups read the norm while others scale the value it is stored in."""
    n = 50 * 4 // size
    other = (8 * BASE, 9 * BASE, 7, B.MOE_F32)
    norm = BASE + 4 * word
    assert lib.moe_grad_clip(pack(other, (BASE, BASE, n, dtype)), 2, norm, 1.0, None) == BAD
    assert lib.moe_grad_clip(pack((2 * BASE, BASE, n, dtype), other), 2, norm, 1.0, None) == BAD


@pytest.mark.parametrize("dtype,size", [(B.MOE_F32, 4), (B.MOE_BF16, 2)])
@pytest.mark.parametrize("word", [0, 25, 49])
def test_the_norm_may_not_be_written_into_a_gradient(lib, dtype, size, word):
    n = 50 * 4 // size
    rows = pack((8 * BASE, 9 * BASE, 7, B.MOE_F32), (BASE, 2 * BASE, n, dtype))
    assert lib.moe_grad_norm(rows, 2, BASE + 4 * word, 5 * BASE, 1 << 40, None) == BAD


def test_a_norm_beside_empty_tensors_is_taken(lib):
    rows = pack((BASE, BASE, 0, B.MOE_F32), (BASE - 8, BASE - 8, 0, B.MOE_BF16))
    assert lib.moe_grad_clip(rows, 2, BASE, 1.0, None) == B.MOE_OK
