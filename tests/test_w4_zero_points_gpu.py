"""Zero points over the whole range that packing takes, 0 .. 63."""
import pytest
import torch

import unstructured_sparse_skinny_b200 as fs
from tests.test_w4_gpu import TYPES, dense64, gen

pytestmark = pytest.mark.gpu


def wide(shape, group, dtype, seed):
    g = gen(seed)
    per = (*shape[:-1], -(-shape[-1] // group))
    codes = torch.randint(0, 16, shape, dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.exp2(torch.randint(-2, 2, per, device="cuda", generator=g).float()).to(dtype)
    return codes, scales, torch.randint(0, 64, per, dtype=torch.uint8, device="cuda", generator=g)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", [(37, 203), (2, 19, 264)])
def test_decode(dtype, group, shape):
    codes, scales, zeros = wide(shape, group, dtype, 1)
    A = fs.w4_pack(codes, scales, zeros, group=group)
    assert torch.equal(fs.w4_decode(A, torch.float32).double(), dense64(codes, scales, zeros, group))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,K,N", [(70, 203, 1), (70, 203, 9), (2600, 8203, 20), (2600, 8203, 140)])
def test_product_is_exact(dtype, group, M, K, N):
    """Activations of -1, 0 and 1 and scales of 1/4 .. 2: sums of multiples of 1/4 below 2^21, so exact in fp32 in any
    order; a weight has 6 bits, which 16-bit types hold."""
    codes, scales, zeros = wide((M, K), group, dtype, K)
    A = fs.w4_pack(codes, scales, zeros, group=group)
    B = torch.randint(-1, 2, (N, K), device="cuda", generator=gen(N)).to(dtype)
    C = torch.empty((N, M), device="cuda")
    assert torch.equal(fs.w4_matmul(A, B, C).double(), B.double() @ dense64(codes, scales, zeros, group).t())


@pytest.mark.parametrize("N", [3, 20, 140])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_padding_never_overflows_alone(N, group):
    """The last column's weights are -5000, which fp16 holds; its group ends there, and what fills the group up must not
    be a weight that fp16 does not hold (infinity times the padding's zero activations)."""
    M, K = 2600, 8193
    codes = torch.full((M, K), 15, dtype=torch.uint8, device="cuda")
    G = -(-K // group)
    scales = torch.ones((M, G), device="cuda", dtype=torch.float16)
    scales[:, -1] = 5000
    zeros = torch.full((M, G), 16, dtype=torch.uint8, device="cuda")
    A = fs.w4_pack(codes, scales, zeros, group=group)
    B = torch.zeros((N, K), device="cuda", dtype=torch.float16)
    B[:, -1] = 2
    B[:, 0] = 1
    assert (fs.w4_matmul(A, B) == -10000).all()  # fp16 has steps of 8 there
    C = torch.empty((N, M), device="cuda")
    assert (fs.w4_matmul(A, B, C) == -10001).all()
