"""An output that overlaps the activations is refused: the product reads them while it writes."""
import pytest
import torch

import unstructured_sparse_skinny_b200 as fs
from unstructured_sparse_skinny_b200.w4 import _overlap


def overlap(a, b):
    return _overlap(a, a.stride(0), b, b.stride(0))


def shares(a, b):
    """By marking a's values."""
    for t in (a, b):
        t.fill_(1)
    a.fill_(0)
    return bool((b == 0).any())


def test_by_marking():
    """All placements of rows in one buffer: what shares memory is found, and equal distances never raise a false alarm."""
    flat = torch.zeros(400, dtype=torch.int16)
    for rows in (1, 2, 5):
        for wa, wb, pa, pb in ((8, 8, 8, 8), (8, 4, 20, 20), (3, 5, 9, 9), (6, 2, 11, 11), (4, 4, 7, 11), (10, 10, 30, 30)):
            for at in range(0, 160, 3):
                for bt in (0, 1, 7, 8, 40, 47, 48, 100, 160):
                    a = flat.as_strided((rows, wa), (pa, 1), at)
                    b = flat.as_strided((rows, wb), (pb, 1), bt)
                    got, want = overlap(a, b), shares(a, b)
                    assert got or not want, (rows, wa, wb, pa, pb, at, bt)
                    if pa == pb or rows == 1:
                        assert got == want, (rows, wa, wb, pa, pb, at, bt)


def test_types_of_different_width():
    flat = torch.zeros(64, dtype=torch.float32)
    half = flat.view(torch.float16)
    B = half.as_strided((4, 6), (32, 1), 0)
    assert not overlap(B, flat.as_strided((4, 13), (16, 1), 3))  # the rest of each 64-byte row
    assert overlap(B, flat.as_strided((4, 13), (16, 1), 2))
    assert not overlap(B[:0], flat.as_strided((0, 13), (16, 1), 0))


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 5, 20, 140])
def test_product(N):
    M = K = 2048
    g = torch.Generator(device="cuda").manual_seed(N)
    A = fs.w4_encode(torch.randn((M, K), device="cuda", generator=g).half())
    both = torch.randn((N, K + M), device="cuda", generator=g).half()
    B = both[:, :K]
    with pytest.raises(ValueError):
        fs.w4_matmul(A, B, B)
    with pytest.raises(ValueError):
        fs.w4_matmul(A, B, both[:, K - 1:K - 1 + M])
    want = fs.w4_matmul(A, B.clone())
    before = B.clone()
    assert torch.equal(fs.w4_matmul(A, B, both[:, K:]), want)  # beside them in the same rows
    assert torch.equal(B, before)
