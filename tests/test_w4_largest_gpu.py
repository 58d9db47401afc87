"""Activations near the end of bf16's range: a product is infinite only where its terms or its sum are."""
import pytest
import torch

import unstructured_sparse_skinny_b200 as fs
from tests.test_w4_gpu import dense64, gen

pytestmark = pytest.mark.gpu


def small_weights(shape, group, seed):
    """Weights of 2^-20 times a whole number."""
    g = gen(seed)
    per = (*shape[:-1], -(-shape[-1] // group))
    codes = torch.randint(0, 16, shape, dtype=torch.uint8, device="cuda", generator=g)
    zeros = torch.randint(0, 64, per, dtype=torch.uint8, device="cuda", generator=g)
    return codes, torch.full(per, 2.0 ** -20, device="cuda", dtype=torch.bfloat16), zeros


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,K,N", [(64, 384, 1), (64, 384, 8), (64, 384, 20), (2600, 8200, 20), (2600, 8200, 140)])
def test_product(M, K, N, group):
    """Every activation is 2^127 (half of the largest) or its negative: whole numbers below 2^20 times 2^107."""
    codes, scales, zeros = small_weights((M, K), group, 1)
    A = fs.w4_pack(codes, scales, zeros, group=group)
    B = torch.randint(0, 2, (N, K), device="cuda", generator=gen(2)).double().mul(2).sub(1).mul(2.0 ** 127).bfloat16()
    B[0] = B[0].abs()  # a row without cancellation
    C = torch.empty((N, M), device="cuda")
    fs.w4_matmul(A, B, C)
    assert torch.equal(C.double(), B.double() @ dense64(codes, scales, zeros, group).t())


@pytest.mark.parametrize("T", [1, 5, 20, 64])
def test_experts(T):
    """gate is 2^-126 x a whole number of at most 2^6, so h is small again and the layer's output finite."""
    E, H, F, group = 3, 256, 128, 64
    codes, _, zeros = small_weights((E, F, H), group, 3)
    scales = torch.full((E, F, H // group), 2.0 ** -120, device="cuda", dtype=torch.bfloat16)
    gate = fs.w4_pack(codes, scales, zeros, group=group)
    down = fs.w4_pack(*small_weights((E, H, F), group, 4), group=group)
    X = torch.full((T, H), 2.0 ** 127, device="cuda", dtype=torch.bfloat16)
    X[:, 1::2] *= -1
    ids = (torch.arange(T, device="cuda", dtype=torch.int32) % E).unsqueeze(1)
    out = fs.moe_w4_experts(X, ids, torch.ones((T, 1), device="cuda"), gate, None, down, activation="relu")
    g, d = dense64(codes, scales, zeros, group), fs.w4_decode(down, torch.float32).double()
    for t in range(T):
        e = int(ids[t])
        h = (g[e] @ X[t].double()).clamp(min=0)  # a whole number times 2^7: below 2^14 steps, so h is exact in two bf16
        want = d[e] @ h
        assert torch.isfinite(out[t]).all()
        # h has 13 bits, the sums are exact, and the output is rounded once
        assert ((out[t].double() - want).abs() <= torch.finfo(torch.bfloat16).eps / 2 * want.abs()).all()


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("M,K,N", [(64, 392, 1), (64, 392, 20), (2600, 8200, 140)])
def test_smallest(M, K, N, group):
    """At the other end sums of a few tokens are held 2^-13 times as large, down to fp32's smallest step of 2^-149: each of
    the K / 16 + 64 additions is off by 2^-23 of the terms or by 2^-136."""
    g = gen(5)
    codes = torch.randint(0, 16, (M, K), dtype=torch.uint8, device="cuda", generator=g)
    scales = (torch.rand((M, -(-K // group)), device="cuda", generator=g) + 0.5).bfloat16()
    A = fs.w4_pack(codes, scales, None, group=group)
    W = dense64(codes, scales, None, group)
    for e in (-60, -100, -120):
        B = torch.randn((N, K), device="cuda", generator=g).double().mul(2.0 ** e).bfloat16()
        C = torch.empty((N, M), device="cuda")
        fs.w4_matmul(A, B, C)
        size = B.double().abs() @ W.abs().t()
        bound = (K / 16 + 64) * (2.0 ** -23 * size + 2.0 ** -136)
        if N > 8:
            bound += 2.0 ** -8 * size  # weights may be rounded
        assert ((C.double() - B.double() @ W.t()).abs() <= bound).all()
