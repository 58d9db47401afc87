"""The skinny product on each of its two kernels, at sizes that the rule sends there."""
import pytest
import torch

import unstructured_sparse_skinny_b200 as fs
from tests.test_w4_gpu import TYPES, codes_of, dense64, gen
from unstructured_sparse_skinny_b200 import binding

pytestmark = pytest.mark.gpu


def on_tensor_memory(A, N):
    """Whether a product with 16-bit output runs on the tensor-memory kernel: for rows on 16 bytes the other one needs no scratch."""
    return binding.load_library().flashspmm_w4_matmul_workspace_bytes(A._ref, 1 << 20, (A.K + 7) // 8 * 8, N) > 0 and \
        A.K % 8 == 0


@pytest.mark.parametrize("M,K,N", [(4096, 8192, 16), (4096, 4096, 24), (2048, 4096, 64)])
@pytest.mark.parametrize("group", [32, 128])
def test_the_same_bits_wherever_the_activations_lie(M, K, N, group):
    codes, scales, zeros = codes_of((M, K), group, torch.bfloat16, False, 3)
    A = fs.w4_pack(codes, scales, zeros, group=group)
    B = torch.randn((N, K), device="cuda", generator=gen(4)).bfloat16()
    want = fs.w4_matmul(A, B)
    wide = torch.zeros((N, K + 3), device="cuda", dtype=torch.bfloat16)
    wide[:, 1:1 + K] = B
    assert torch.equal(fs.w4_matmul(A, wide[:, 1:1 + K]), want)
