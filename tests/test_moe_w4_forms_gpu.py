"""The experts' kernels in every form: zero points in each of the three stacks, with and without the gate product, and
each number of tokens that an expert's records serve at a time (8, 16 and 32)."""
import pytest
import torch

import unstructured_sparse_skinny_b200 as fs
from tests.test_moe_w4_gpu import check, experts64
from tests.test_w4_gpu import TYPES, codes_of, dense64, gen

pytestmark = pytest.mark.gpu


def stacks(E, H, F, group, dtype, symmetric, up):
    dense, packed = [], []
    for i, shape in enumerate(((E, F, H), (E, F, H), (E, H, F))):
        codes, scales, zeros = codes_of(shape, group, dtype, symmetric[i], 10 + i)
        dense.append(dense64(codes, scales, zeros, group))
        packed.append(fs.w4_pack(codes, scales, zeros, group=group))
    if not up:
        dense[1] = packed[1] = None
    return dense, packed


# tokens, experts: up to 8 tokens; 16 at a time; 32 at a time (more than 12 tokens an expert on average)
@pytest.mark.parametrize("T,E", [(5, 4), (14, 4), (40, 12), (40, 3)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [(False, False, False), (True, False, True), (False, True, False), (True, True, False)])
@pytest.mark.parametrize("up", [True, False])
def test_forms(T, E, group, symmetric, up):
    H, F, k, dtype = 392, 328, 2, TYPES[(T + group) % 2]
    dense, packed = stacks(E, H, F, group, dtype, symmetric, up)
    X = torch.randn((T, H), device="cuda", generator=gen(T)).to(dtype)
    ids = torch.stack([torch.randperm(E, device="cuda", generator=gen(t))[:k] for t in range(T)]).int()
    weights = torch.rand((T, k), device="cuda", generator=gen(2))
    act = ("silu", "gelu", "relu")[(T + E) % 3]
    out = fs.moe_w4_experts(X, ids, weights, *packed, activation=act)
    check(out, *experts64(X, ids, weights, dense, act, dtype))


@pytest.mark.parametrize("T", [6, 12, 50])
@pytest.mark.parametrize("dtype", TYPES)
def test_zero_points_up_to_63(T, dtype):
    E, H, F, group, k = 3, 264, 200, 64, 1
    g, parts = gen(4), []
    for shape in ((E, F, H), (E, F, H), (E, H, F)):
        codes, scales, zeros = codes_of(shape, group, dtype, False, 6)
        parts.append((codes, scales, torch.randint(0, 64, zeros.shape, dtype=torch.uint8, device="cuda", generator=g)))
    dense = [dense64(*p, group) for p in parts]
    packed = [fs.w4_pack(*p, group=group) for p in parts]
    X = torch.randn((T, H), device="cuda", generator=g).to(dtype) * 0.1
    ids = (torch.arange(T, device="cuda", dtype=torch.int32) % E).unsqueeze(1)
    weights = torch.rand((T, k), device="cuda", generator=g)
    check(fs.moe_w4_experts(X, ids, weights, *packed), *experts64(X, ids, weights, dense, "silu", dtype))


@pytest.mark.parametrize("T", [1, 40])
def test_in_place(T):
    """The output may take the activations' place."""
    E, H, F, k = 4, 256, 128, 2
    _, packed = stacks(E, H, F, 64, torch.float16, (False, ) * 3, True)
    router = torch.randn((E, H), device="cuda", generator=gen(3))
    X = torch.randn((T, H), device="cuda", generator=gen(T)).half()
    want, _, _ = fs.moe_w4(X, router, *packed, k)
    out, _, _ = fs.moe_w4(X, router, *packed, k, out=X)
    assert out is X and torch.equal(X, want)


def test_captured_behind_a_copy():
    """In a graph the first kernel may follow a node that is no kernel."""
    E, H, F, k, T = 8, 256, 128, 2, 4
    _, packed = stacks(E, H, F, 64, torch.bfloat16, (False, ) * 3, True)
    router = torch.randn((E, H), device="cuda", generator=gen(3)).bfloat16()
    source = torch.randn((T, H), device="cuda", generator=gen(1)).bfloat16()
    X = torch.zeros_like(source)
    want = fs.moe_w4(source, router, *packed, k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        X.copy_(source)
        got = fs.moe_w4(X, router, *packed, k)
    for _ in range(3):
        X.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
