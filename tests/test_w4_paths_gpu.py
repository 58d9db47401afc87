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


def check(got, W, B, rounded_weights):
    """Bound of one output: (K / 16 + 64) * 2^-23 * sum |w x| for the sums, as in test_w4_gpu.py, eps / 2 of sum |w x|
    where weights are rounded to 16 bits, eps / 2 of the value for a 16-bit output and half its smallest step."""
    want, size = B.double() @ W.t(), B.double().abs() @ W.abs().t()
    eps, K = torch.finfo(B.dtype).eps, W.shape[1]
    bound = (K / 16 + 64) * 2.0 ** -23 * size
    if rounded_weights:
        bound += eps / 2 * size
    if got.dtype is not torch.float32:
        bound += eps / 2 * (want.abs() + bound) + torch.finfo(B.dtype).smallest_normal * eps
    off = (got.double() - want).abs()
    assert (off <= bound).all(), f"{(off / bound).max().item():.3g} of the bound"
    # Roundings of weights are independent: over a row of K they add up like their root of squares, and a whole result
    # is no further off than one rounding of the output (eps / 2) and one of the weights (eps / 2).
    assert off.norm() <= (eps + 1e-6) * want.norm()


M, K = 2600, 8200  # 21 blocks of 65 units: shared and whole blocks, a last block of 40 rows and a last unit of 8 columns


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("N", [33, 64, 65, 100, 128, 129, 200, 256])
def test_tensor_memory_kernel(dtype, group, symmetric, N):
    codes, scales, zeros = codes_of((M, K), group, dtype, symmetric, N)
    A = fs.w4_pack(codes, scales, zeros, group=group)
    assert on_tensor_memory(A, N)
    B = torch.randn((N, K), device="cuda", generator=gen(N)).to(dtype)
    check(fs.w4_matmul(A, B), dense64(codes, scales, zeros, group), B, True)


@pytest.mark.parametrize("group,symmetric", [(32, False), (64, True), (128, False)])
@pytest.mark.parametrize("rows,columns,N", [(129, 65536, 40), (12288, 1032, 100), (40000, 136, 70), (128, 33000, 256),
                                            (4099, 5008, 17), (12288, 4104, 12)])
def test_tensor_memory_kernel_shapes(rows, columns, N, group, symmetric):
    """Few rows and many columns, the other way round, and the fewest tokens that go there."""
    codes, scales, zeros = codes_of((rows, columns), group, torch.bfloat16, symmetric, N)
    A = fs.w4_pack(codes, scales, zeros, group=group)
    B = torch.randn((N, columns), device="cuda", generator=gen(N)).bfloat16()
    check(fs.w4_matmul(A, B), dense64(codes, scales, zeros, group), B, on_tensor_memory(A, N))


@pytest.mark.parametrize("N", [40, 140])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_tensor_memory_kernel_strides(N, group):
    codes, scales, zeros = codes_of((M, K), group, torch.float16, False, 2)
    A = fs.w4_pack(codes, scales, zeros, group=group)
    assert on_tensor_memory(A, N)
    B = torch.randn((N, K), device="cuda", generator=gen(1)).half()
    want = fs.w4_matmul(A, B)
    for pitch, first in ((K + 8, 8), (K + 3, 1), (K + 1, 0), (K + 5, 5)):
        wide = torch.full((N, pitch), float("nan"), device="cuda", dtype=torch.float16)
        wide[:, first:first + K] = B
        assert torch.equal(fs.w4_matmul(A, wide[:, first:first + K]), want)
    assert torch.equal(fs.w4_matmul(A, B[:1].expand(N, K)), want[:1].expand(N, M))
    wide = torch.full((N + 2, M + 9), 5.0, device="cuda", dtype=torch.float16)
    fs.w4_matmul(A, B, wide[1:N + 1, 4:4 + M])
    assert torch.equal(wide[1:N + 1, 4:4 + M], want)
    wide[1:N + 1, 4:4 + M] = 5
    assert (wide == 5).all()


@pytest.mark.parametrize("N", [40, 140])
@pytest.mark.parametrize("group", [32, 128])
def test_tensor_memory_kernel_non_finite_activations(N, group):
    codes, scales, zeros = codes_of((M, K), group, torch.float16, True, 2)
    codes[:, 5] = 9  # no weight of column 5 is zero
    A = fs.w4_pack(codes, scales, zeros, group=group)
    assert on_tensor_memory(A, N)
    B = torch.randn((N, K), device="cuda", generator=gen(1)).half()
    want = fs.w4_matmul(A, B)
    for value in (float("inf"), -float("inf"), float("nan")):
        B[N - 1, 5] = value
        got = fs.w4_matmul(A, B)
        assert torch.equal(got[:-1], want[:-1])
        assert torch.isnan(got[-1]).all() if value != value else (got[-1] == value).all()


@pytest.mark.parametrize("N", [40, 140])
def test_tensor_memory_kernel_non_finite_scales(N):
    """A row with a scale that is not finite is not finite, and the others are as they were."""
    codes, scales, zeros = codes_of((M, K), 64, torch.bfloat16, False, 2)
    B = torch.randn((N, K), device="cuda", generator=gen(1)).bfloat16()
    want = fs.w4_matmul(fs.w4_pack(codes, scales, zeros, group=64), B)
    scales[77, 3], scales[2590, 128] = float("inf"), float("nan")
    got = fs.w4_matmul(fs.w4_pack(codes, scales, zeros, group=64), B)
    assert not torch.isfinite(got[:, [77, 2590]]).any()
    got[:, [77, 2590]] = want[:, [77, 2590]]
    assert torch.equal(got, want)


@pytest.mark.parametrize("N", [40, 140])
@pytest.mark.parametrize("group", [32, 128])
def test_tensor_memory_kernel_in_graphs_and_streams(N, group):
    """A captured call and eager ones, on two streams, at once."""
    codes, scales, zeros = codes_of((M, K), group, torch.bfloat16, False, 2)
    A = fs.w4_pack(codes, scales, zeros, group=group)
    assert on_tensor_memory(A, N)
    Bs = [torch.randn((N, K), device="cuda", generator=gen(i)).bfloat16() for i in range(3)]
    want = [fs.w4_matmul(A, b) for b in Bs]
    x, graph, side = Bs[0].clone(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        out = fs.w4_matmul(A, x)
    for i in (1, 2, 0):
        x.copy_(Bs[i])
        torch.cuda.synchronize()
        graph.replay()
        other = [fs.w4_matmul(A, b, stream=side) for b in Bs]
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]) and all(torch.equal(a, b) for a, b in zip(other, want))


# ---------------------------------------------------------------- fp32 output: no weight is rounded

def launches(call):
    before = fs.launch_count()
    call()
    return fs.launch_count() - before


def check32(C, W, B):
    """Sums over the weights and over their rests, 2 K / 16 steps of the tensor cores, and nothing else."""
    want, size = B.double() @ W.t(), B.double().abs() @ W.abs().t()
    bound = (2 * W.shape[1] / 16 + 64) * 2.0 ** -23 * size
    off = (C.double() - want).abs()
    assert (off <= bound).all(), f"{(off / bound).max().item():.3g} of the bound"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("N", [48, 64, 100, 128, 129, 256])
def test_fp32_output(dtype, group, symmetric, N):
    codes, scales, zeros = codes_of((M, K), group, dtype, symmetric, N)
    A = fs.w4_pack(codes, scales, zeros, group=group)
    B = torch.randn((N, K), device="cuda", generator=gen(N)).to(dtype)
    C = torch.empty((N, M), device="cuda")
    assert launches(lambda: fs.w4_matmul(A, B, C)) == 2  # rows on 16 bytes: one launch is fragments
    check32(C, dense64(codes, scales, zeros, group), B)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("rows,columns,N", [(129, 65536, 40), (12288, 1032, 100), (40000, 136, 70), (128, 33001, 256),
                                            (4099, 5003, 17), (1, 1, 256), (130, 120, 9), (8192, 8195, 24)])
def test_fp32_output_shapes(rows, columns, N, group):
    codes, scales, zeros = codes_of((rows, columns), group, torch.float16, False, N)
    A = fs.w4_pack(codes, scales, zeros, group=group)
    B = torch.randn((N, columns), device="cuda", generator=gen(N)).half()
    C = torch.empty((N, rows), device="cuda")
    check32(fs.w4_matmul(A, B, C), dense64(codes, scales, zeros, group), B)


@pytest.mark.parametrize("N", [48, 140])
@pytest.mark.parametrize("dtype", TYPES)
def test_fp32_output_over_the_range_of_scales(N, dtype):
    """Rests of the smallest weights are whole steps of the type, and weights up to twice the largest value are exact."""
    codes, _, zeros = codes_of((M, K), 64, dtype, False, 1)
    fin = torch.finfo(dtype)
    g = gen(3)
    for low, high in ((fin.smallest_normal / 8, fin.smallest_normal * 4), (1e-3, 1e-2), (fin.max / 16, fin.max / 8)):
        scales = (torch.rand((M, -(-K // 64)), device="cuda", generator=g).double() * (high - low) + low).to(dtype)
        B = torch.randn((N, K), device="cuda", generator=g)
        # sums of K weights of fin.max stay finite in bf16, and the smallest ones above fp32's own steps
        B = (B * 2.0 ** -20 if high > 1 else B * 2.0 ** 20 if high < 1e-30 else B).to(dtype)
        A = fs.w4_pack(codes, scales, zeros, group=64)
        C = torch.empty((N, M), device="cuda")
        check32(fs.w4_matmul(A, B, C), dense64(codes, scales, zeros, 64), B)


@pytest.mark.parametrize("N", [48, 140])
@pytest.mark.parametrize("dtype", TYPES)
def test_fp32_output_of_non_finite_activations(N, dtype):
    codes, scales, zeros = codes_of((M, K), 32, dtype, True, 2)
    codes[:, 5] = 9  # no weight of column 5 is zero; many of its rests are
    A = fs.w4_pack(codes, scales, zeros, group=32)
    B = torch.randn((N, K), device="cuda", generator=gen(1)).to(dtype)
    want = fs.w4_matmul(A, B, torch.empty((N, M), device="cuda"))
    for value in (float("inf"), -float("inf"), float("nan")):
        for column in (5, 4):
            B[N - 1, column] = value
            got = fs.w4_matmul(A, B, torch.empty((N, M), device="cuda"))
            assert torch.equal(got[:-1], want[:-1])
            if column == 5:
                assert torch.isnan(got[-1]).all() if value != value else (got[-1] == value).all()
                B[N - 1, 5] = 1
            else:  # weights of both signs and zero
                w = dense64(codes, scales, zeros, 32)[:, 4]
                assert torch.equal(torch.nan_to_num(got[-1].double(), nan=7, posinf=8, neginf=9),
                                   torch.nan_to_num(w * value, nan=7, posinf=8, neginf=9))
                B[N - 1, 4] = 1


@pytest.mark.parametrize("N", [48, 140])
def test_fp32_output_of_non_finite_scales(N):
    codes, scales, zeros = codes_of((M, K), 64, torch.bfloat16, False, 2)
    B = torch.randn((N, K), device="cuda", generator=gen(1)).bfloat16()
    want = fs.w4_matmul(fs.w4_pack(codes, scales, zeros, group=64), B, torch.empty((N, M), device="cuda"))
    scales[77, 3], scales[2590, 128] = float("inf"), float("nan")
    got = fs.w4_matmul(fs.w4_pack(codes, scales, zeros, group=64), B, torch.empty((N, M), device="cuda"))
    assert not torch.isfinite(got[:, [77, 2590]]).any()
    got[:, [77, 2590]] = want[:, [77, 2590]]
    assert torch.equal(got, want)


@pytest.mark.parametrize("N", [48, 140])
def test_fp32_output_strides_and_graphs(N):
    codes, scales, zeros = codes_of((M, K), 128, torch.float16, False, 2)
    A = fs.w4_pack(codes, scales, zeros)
    B = torch.randn((N, K), device="cuda", generator=gen(1)).half()
    want = fs.w4_matmul(A, B, torch.empty((N, M), device="cuda"))
    wide = torch.full((N, K + 3), float("nan"), device="cuda", dtype=torch.float16)
    wide[:, 1:1 + K] = B
    out = torch.full((N, M + 9), 5.0, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fs.w4_matmul(A, wide[:, 1:1 + K], out[:, 4:4 + M])
    for _ in range(3):
        out[:, 4:4 + M] = 5
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:, 4:4 + M], want) and (out[:, :4] == 5).all() and (out[:, 4 + M:] == 5).all()
