"""Sizes at the end of their ranges, without a GPU: byte counts that pass 63 bits are refused, not wrapped."""
import ctypes

import pytest

from unstructured_sparse_skinny_b200 import binding
from unstructured_sparse_skinny_b200.build import build_library
from unstructured_sparse_skinny_b200.w4 import _W4View

FAKE = 0x7F0000000000
UNSUPPORTED = 2


@pytest.fixture(scope="module")
def lib():
    build_library()
    return binding.load_library()


@pytest.mark.parametrize("group,zeros", [(128, 0), (32, 1)])
@pytest.mark.parametrize("M,K", [(1 << 30, 1 << 30), (1 << 30, 1000), (77, 1 << 30), (1, 1)])
@pytest.mark.parametrize("count", [1, 2, 7, 8, 15, 16, 17, 31, 32, 64, 1 << 20, (1 << 31) - 1])
def test_bytes(lib, M, K, count, group, zeros):
    record = 1024 + 16 * (128 // group) * (3 if zeros else 2)
    exact = count * -(-M // 128) * 8 * -(-K // 128) * record
    want = exact if exact < 1 << 63 else -1
    assert lib.flashspmm_w4_bytes(M, K, count, group, zeros) == want
    if want < 0:
        v = ctypes.byref(_W4View(M, K, count, group, 0, zeros, FAKE))
        assert lib.flashspmm_w4_decode(v, FAKE, 0, None) == UNSUPPORTED
        assert lib.flashspmm_w4_encode(FAKE, K, 1 - zeros, v, None) == UNSUPPORTED
