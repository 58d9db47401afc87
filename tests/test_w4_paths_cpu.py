"""Which of its two kernels a product runs on, seen from the size of its scratch: none for rows on 16 bytes on
fragments, an image of the activations on the tensor-memory kernel."""
import ctypes

import pytest

from unstructured_sparse_skinny_b200 import binding
from unstructured_sparse_skinny_b200.build import build_library
from unstructured_sparse_skinny_b200.w4 import _W4View

FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    build_library()
    return binding.load_library()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,K", [(2048, 2048), (4096, 4096), (4096, 8192), (6000, 5000), (9216, 9216), (16384, 16384)])
def test_the_kernel_depends_on_sizes_alone(lib, M, K, group):
    """Activations elsewhere in memory, or further apart, run on the same kernel: the same bits come out."""
    A = ctypes.byref(_W4View(M, K, 1, group, 0, 0, FAKE))
    for N in (1, 8, 9, 12, 16, 17, 24, 32, 33, 40, 64, 100, 128, 200, 256):
        need = lib.flashspmm_w4_matmul_workspace_bytes(A, FAKE, K, N)
        for at, ldb in ((FAKE + 2, K), (FAKE, K + 1), (FAKE + 8, K + 4)):
            copied = N * K * 2  # what fragments need for rows that are not on 16 bytes (K % 8 == 0 here)
            assert lib.flashspmm_w4_matmul_workspace_bytes(A, at, ldb, N) == (need or copied), N
