"""4-bit weights on the GPU: encoder, packing, decoder and the skinny product
against plain fp64 forms.

Where the values allow it the comparison is exact: with scales that are powers
of two and small whole activations every sum below 2^24 is a whole number that
fp32 holds, whatever the order.  Elsewhere the bound counts roundings:

  half a step of the output type, eps / 2 of the value;
  one rounding (or truncation) of at most 2^-23 of the running sum for each
  tensor-core step of 16 columns and for each of the few dozen additions that
  join groups, warps and splits: (K / 16 + 64) * 2^-23 * sum |w x|;
  where the weight itself is rounded to 16 bits before the product (N > 8, as
  the header says), eps / 2 of sum |w x|.
"""
import pytest
import torch

import unstructured_sparse_skinny_b200 as fs

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes_of(shape, group, dtype, symmetric, seed, whole=False):
    g = gen(seed)
    per = (*shape[:-1], -(-shape[-1] // group))
    codes = torch.randint(0, 16, shape, dtype=torch.uint8, device="cuda", generator=g)
    if whole:
        scales = torch.exp2(torch.randint(-2, 3, per, device="cuda", generator=g).float()).to(dtype)
    else:
        scales = (torch.rand(per, device="cuda", generator=g) * 0.01 + 0.001).to(dtype)
    zeros = None if symmetric else torch.randint(0, 16, per, dtype=torch.uint8, device="cuda", generator=g)
    return codes, scales, zeros


def dense64(codes, scales, zeros, group):
    K = codes.shape[-1]
    col = torch.arange(K, device=codes.device) // group
    z = 8.0 if zeros is None else zeros.double()[..., col]
    return (codes.double() - z) * scales.double()[..., col]


def encode64(W, group, symmetric):
    """The encoder's definition: (codes, scales, zeros), roundings to even."""
    M, K = W.shape
    G = -(-K // group)
    w = torch.nn.functional.pad(W.double(), (0, G * group - K)).view(M, G, group)
    if symmetric:
        s = (w.abs().amax(-1) / 7).to(W.dtype)
        z = torch.full((M, G), 8.0, dtype=torch.float64, device=W.device)
    else:
        low, high = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
        s = ((high - low) / 15).to(W.dtype)
        d = s.double()
        z = torch.where(d > 0, (-low / torch.where(d > 0, d, 1.0)).round(), (-low).round()).clamp(0, 15)
    d = torch.where(s > 0, s.double(), 1.0)
    q = ((w / d.unsqueeze(-1)).round() + z.unsqueeze(-1)).clamp(0, 15)
    return q.view(M, G * group)[:, :K], s, z


# ---------------------------------------------------------------- format

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("shape", [(1, 1), (16, 128), (37, 200), (130, 131), (2, 19, 264)])
def test_pack_decode_is_exact(dtype, group, symmetric, shape):
    codes, scales, zeros = codes_of(shape, group, dtype, symmetric, 1)
    A = fs.w4_pack(codes, scales, zeros, group=group)
    want = dense64(codes, scales, zeros, group)
    assert torch.equal(fs.w4_decode(A, torch.float32).double(), want)
    assert torch.equal(fs.w4_decode(A), want.to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("M,K", [(1, 1), (16, 128), (50, 328), (33, 331)])
def test_encode_follows_its_definition(dtype, group, symmetric, M, K):
    g = gen(M + K)
    W = (torch.randn((M, K), device="cuda", generator=g) * 0.05).to(dtype)
    W[:, : K // 3] = (W[:, : K // 3].float() * 64).round().div(64).to(dtype)  # many values half way between codes
    W[M // 2] = 0
    A = fs.w4_encode(W, group=group, symmetric=symmetric)
    q, s, z = encode64(W, group, symmetric)
    col = torch.arange(K, device="cuda") // group
    want = (q - z[:, col]) * s.double()[:, col]
    assert torch.equal(fs.w4_decode(A, torch.float32).double(), want)
    assert (fs.w4_decode(A)[M // 2] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_encode_ties_go_to_even(dtype):
    W = torch.zeros((1, 32), device="cuda", dtype=dtype)
    W[0, :8] = torch.tensor([7.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, -7.0])  # s = 1
    got = fs.w4_decode(fs.w4_encode(W, group=32), torch.float32)[0, :8]
    assert got.tolist() == [7, 0, 2, 2, 0, -2, -2, -7]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("symmetric", [True, False])
def test_encode_range_of_scales(dtype, symmetric):
    """Groups at both ends of the type's range, down to scales that round to zero or are not normal numbers."""
    fin = torch.finfo(dtype)
    sizes = [fin.max, fin.tiny * 15, fin.tiny, fin.smallest_normal / 4, 1e-30 if dtype is torch.bfloat16 else 1e-3]
    g = gen(5)
    W = torch.cat([(torch.rand((3, 32), device="cuda", generator=g).double() * 2 - 1).mul(s).to(dtype) for s in sizes])
    A = fs.w4_encode(W, group=32, symmetric=symmetric)
    q, s, z = encode64(W, 32, symmetric)
    # 8 * s may pass the largest fp32 value: the decoder's value is the exact one rounded to fp32
    assert torch.equal(fs.w4_decode(A, torch.float32), ((q - z) * s.double()).float())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("symmetric", [True, False])
def test_encode_keeps_non_finite_groups_non_finite(bad, symmetric):
    W = torch.randn((20, 256), device="cuda", generator=gen(3)).half()
    clean = fs.w4_decode(fs.w4_encode(W, symmetric=symmetric))
    W[4, 130] = bad
    got = fs.w4_decode(fs.w4_encode(W, symmetric=symmetric))
    assert not torch.isfinite(got[4, 128:]).any()
    got[4, 128:] = clean[4, 128:]
    assert torch.equal(got, clean)


def test_encode_strided_rows_and_stacks():
    W = torch.randn((40, 300), device="cuda", generator=gen(4)).half()
    whole = fs.w4_decode(fs.w4_encode(W[:, :256].contiguous()))
    assert torch.equal(fs.w4_decode(fs.w4_encode(W[:, :256])), whole)       # rows 300 values apart, on 8 bytes only
    assert torch.equal(fs.w4_decode(fs.w4_encode(W.t()[:256].t())), whole)  # the same view
    stack = torch.randn((3, 40, 256), device="cuda", generator=gen(6)).bfloat16()
    A = fs.w4_encode(stack, group=64, symmetric=False)
    got = fs.w4_decode(A)
    for e in range(3):
        one = fs.w4_decode(fs.w4_encode(stack[e], group=64, symmetric=False))
        assert torch.equal(got[e], one) and torch.equal(fs.w4_decode(A.matrix(e)), one)


# ---------------------------------------------------------------- product

def check_product(got, W, B, dtype, what=""):
    want, size = B.double() @ W.t(), B.double().abs() @ W.abs().t()
    K, eps = W.shape[1], torch.finfo(dtype).eps
    bound = (K / 16 + 64) * 2.0 ** -23 * size
    if B.shape[0] > 8:
        bound += eps / 2 * size
    if got.dtype is not torch.float32:
        bound += eps / 2 * (want.abs() + bound) + torch.finfo(dtype).smallest_normal * eps
    off = (got.double() - want).abs()
    assert (off <= bound).all(), f"{what}: {(off / bound).max().item():.3g} of the bound"
    # the roundings are independent, so the whole result is nearer than the sum of the worst cases:
    # one rounding of the output (eps / 2) and one of the weights (eps / 2)
    assert off.norm() <= (eps + 1e-6) * want.norm(), what


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("N", [1, 2, 8, 9, 16, 17, 33, 64, 100, 256])
def test_matmul(dtype, group, symmetric, N):
    M, K = 200 + N, 1000  # neither a whole strip nor a whole unit
    codes, scales, zeros = codes_of((M, K), group, dtype, symmetric, N)
    A = fs.w4_pack(codes, scales, zeros, group=group)
    B = torch.randn((N, K), device="cuda", generator=gen(N)).to(dtype)
    W = dense64(codes, scales, zeros, group)
    check_product(fs.w4_matmul(A, B), W, B, dtype)
    C = torch.empty((N, M), device="cuda")
    assert fs.w4_matmul(A, B, C) is C
    check_product(C, W, B, dtype, "fp32 output")


@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (1, 129, 3), (15, 7, 8), (16, 128, 1), (17, 8, 256), (129, 257, 17),
                                   (4099, 5003, 17), (128, 36864, 5), (20000, 640, 256), (1280, 24576, 256),
                                   (1280, 24576, 200), (20000, 640, 144), (2600, 24576, 24), (8192, 8192, 12), (300, 300, 250), (320, 49152, 70), (9216, 64, 1), (2048, 2048, 40)])
@pytest.mark.parametrize("dtype", TYPES)
def test_matmul_whole_numbers_are_exact(M, K, N, dtype):
    codes, scales, zeros = codes_of((M, K), 64, dtype, False, 7, whole=True)
    A = fs.w4_pack(codes, scales, zeros, group=64)
    B = torch.randint(-1, 2, (N, K), device="cuda", generator=gen(8)).to(dtype)
    want = B.double() @ dense64(codes, scales, zeros, 64).t()
    C = torch.empty((N, M), device="cuda")
    assert torch.equal(fs.w4_matmul(A, B, C).double(), want)
    assert torch.equal(fs.w4_matmul(A, B), want.to(dtype))


@pytest.mark.parametrize("N", [1, 5, 24, 130])
def test_matmul_strides_and_alignment(N):
    M, K = 77, 512
    codes, scales, zeros = codes_of((M, K), 128, torch.float16, False, 2)
    A = fs.w4_pack(codes, scales, zeros)
    B = torch.randn((N, K), device="cuda", generator=gen(1)).half()
    want = fs.w4_matmul(A, B)
    for pitch, shift in ((K + 8, 8), (K + 3, 1), (K + 1, 0)):
        big = torch.full((N, pitch), float("nan"), device="cuda", dtype=torch.float16)
        view = big.flatten()[: N * pitch].view(N, pitch)[:, shift: shift + K] if shift + K <= pitch else None
        view.copy_(B)
        assert torch.equal(fs.w4_matmul(A, view), want)
    flat = torch.empty(N * K + 1, device="cuda", dtype=torch.float16)
    flat[1:].view(N, K).copy_(B)
    assert torch.equal(fs.w4_matmul(A, flat[1:].view(N, K)), want)  # off 16 bytes
    assert torch.equal(fs.w4_matmul(A, B.t().contiguous().t()), want)
    assert torch.equal(fs.w4_matmul(A, B[:1].expand(N, K)), want[:1].expand(N, M))
    big = torch.full((N, M + 9), 5.0, device="cuda", dtype=torch.float16)
    fs.w4_matmul(A, B, big[:, 4: 4 + M])
    assert torch.equal(big[:, 4: 4 + M], want) and (big[:, :4] == 5).all() and (big[:, 4 + M:] == 5).all()


def test_matmul_writes_only_its_rows_and_columns():
    A = fs.w4_pack(*codes_of((40, 128), 128, torch.float16, True, 2))
    B = torch.randn((3, 128), device="cuda", generator=gen(1)).half()
    C = torch.full((8, 40), 7.0, device="cuda", dtype=torch.float16)
    fs.w4_matmul(A, B, C[2:5])
    assert (C[:2] == 7).all() and (C[5:] == 7).all()
    assert torch.equal(C[2:5], fs.w4_matmul(A, B))


@pytest.mark.parametrize("N", [2, 40])
def test_matmul_non_finite_activations_stay_in_their_row(N):
    codes, scales, zeros = codes_of((64, 384), 128, torch.float16, True, 2)
    codes[:, 5] = 9  # no weight of column 5 is zero
    A = fs.w4_pack(codes, scales, zeros)
    B = torch.randn((N, 384), device="cuda", generator=gen(1)).half()
    want = fs.w4_matmul(A, B)
    B[1, 5] = float("inf")
    got = fs.w4_matmul(A, B)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2:], want[2:])
    assert (got[1] == float("inf")).all()
    B[1, 5] = float("nan")
    assert torch.isnan(fs.w4_matmul(A, B)[1]).all()


@pytest.mark.parametrize("N,K", [(3, 131), (200, 4096)])
def test_matmul_checks_its_workspace(N, K):
    """Too small, missing or misaligned scratch is refused and nothing is written."""
    from unstructured_sparse_skinny_b200 import binding
    lib = binding.load_library()
    A = fs.w4_pack(*codes_of((2048, K), 128, torch.float16, True, 2))
    B = torch.ones((N, K), device="cuda", dtype=torch.float16)
    C = torch.full((N, 2048), 5.0, device="cuda", dtype=torch.float16)
    need = lib.flashspmm_w4_matmul_workspace_bytes(A._ref, B.data_ptr(), K, N)
    assert need > 0
    ws = torch.empty(need + 16, device="cuda", dtype=torch.uint8)
    stream = torch.cuda.current_stream().cuda_stream

    def call(ptr, size):
        return lib.flashspmm_w4_matmul(A._ref, B.data_ptr(), K, C.data_ptr(), 2048, 0, N, ptr, size, stream)

    assert call(None, need) == 4 and call(ws.data_ptr(), need - 1) == 4 and call(ws.data_ptr() + 8, need) == 3
    torch.cuda.synchronize()
    assert (C == 5).all()
    assert call(ws.data_ptr(), need) == 0
    assert torch.equal(C, fs.w4_matmul(A, B))


def test_matmul_empty():
    A = fs.w4_pack(*codes_of((40, 128), 128, torch.float16, True, 2))
    assert fs.w4_matmul(A, torch.empty((0, 128), device="cuda", dtype=torch.float16)).shape == (0, 40)
    none = fs.w4_encode(torch.empty((40, 0), device="cuda", dtype=torch.float16))
    big = torch.full((3, 50), 5.0, device="cuda", dtype=torch.float16)
    fs.w4_matmul(none, torch.empty((3, 0), device="cuda", dtype=torch.float16), big[:, :40])
    assert (big[:, :40] == 0).all() and (big[:, 40:] == 5).all()
    rows = fs.w4_encode(torch.empty((0, 64), device="cuda", dtype=torch.float16))
    assert fs.w4_matmul(rows, torch.ones((3, 64), device="cuda", dtype=torch.float16)).shape == (3, 0)


def test_refusals():
    A = fs.w4_pack(*codes_of((40, 128), 128, torch.float16, True, 2))
    B = torch.ones((3, 128), device="cuda", dtype=torch.float16)
    with pytest.raises(TypeError):
        fs.w4_matmul(A, B.bfloat16())
    with pytest.raises(TypeError):
        fs.w4_matmul(A, B.cpu())
    with pytest.raises(ValueError):
        fs.w4_matmul(A, B[:, :64])
    with pytest.raises(ValueError):
        fs.w4_matmul(A, B, torch.empty((3, 41), device="cuda", dtype=torch.float16))
    with pytest.raises(TypeError):
        fs.w4_matmul(A, B, torch.empty((3, 40), device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        fs.w4_matmul(A, B, torch.empty((1, 40), device="cuda", dtype=torch.float16).expand(3, 40))
    with pytest.raises(fs.FlashSpmmError) as e:
        fs.w4_matmul(A, torch.ones((257, 128), device="cuda", dtype=torch.float16))
    assert e.value.status == 2
    with pytest.raises(RuntimeError):
        fs.w4_matmul(A, B.float().requires_grad_().half())
    with pytest.raises(ValueError):
        fs.w4_encode(B, group=16)
    codes, scales, _ = codes_of((40, 128), 128, torch.float16, True, 2)
    with pytest.raises(ValueError):
        fs.w4_pack(codes, scales[:, :0], None)
    with pytest.raises(IndexError):
        A.matrix(1)
    stack = fs.w4_pack(*codes_of((2, 40, 128), 128, torch.float16, True, 2))
    with pytest.raises(fs.FlashSpmmError):
        fs.w4_matmul(stack, B)


@pytest.mark.parametrize("N", [3, 40, 200])
def test_matmul_streams_and_graphs(N):
    """Two streams at once, and a captured call replayed on new activations between eager ones."""
    M, K = 1024, 2051  # the activations are copied to scratch
    codes, scales, zeros = codes_of((M, K), 64, torch.bfloat16, False, 2)
    A = fs.w4_pack(codes, scales, zeros, group=64)
    Bs = [torch.randn((N, K), device="cuda", generator=gen(i)).bfloat16() for i in range(4)]
    want = [fs.w4_matmul(A, b) for b in Bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [fs.w4_matmul(A, Bs[i % 4], stream=streams[i % 2] if i % 4 < 2 else streams[i % 2].cuda_stream)
           for i in range(16)]
    torch.cuda.synchronize()
    assert all(torch.equal(got[i], want[i % 4]) for i in range(16))
    inputs, graphs, outs = [b.clone() for b in Bs[:2]], [], []
    for x in inputs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fs.w4_matmul(A, x))
        graphs.append(g)
    for i in (1, 3):
        inputs[0].copy_(Bs[i])
        inputs[1].copy_(Bs[i - 1])
        graphs[0].replay()
        eager = fs.w4_matmul(A, Bs[2])
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[i]) and torch.equal(outs[1], want[i - 1]) and torch.equal(eager, want[2])


def test_matmul_is_deterministic():
    A = fs.w4_pack(*codes_of((3000, 4096), 128, torch.float16, False, 2))
    for N in (1, 16, 48, 256):
        B = torch.randn((N, 4096), device="cuda", generator=gen(1)).half()
        first = fs.w4_matmul(A, B)
        for _ in range(5):
            assert torch.equal(fs.w4_matmul(A, B), first)


def test_a_layer_runs_on_4_bit_weights_next_to_sparse_ones():
    """Encode a dense layer both ways and chain the two products as a decoder's MLP does."""
    g = gen(9)
    up = (torch.randn((1024, 512), device="cuda", generator=g) * 0.05).half()
    down = (torch.randn((512, 1024), device="cuda", generator=g) * 0.05).half()
    x = torch.randn((8, 512), device="cuda", generator=g).half()
    up4, down4 = fs.w4_encode(up, group=64, symmetric=False), fs.w4_encode(down, group=64, symmetric=False)
    y = fs.w4_matmul(down4, torch.relu(fs.w4_matmul(up4, x)))
    # the same product through the sparse path on the decoded weights
    up_s, down_s = fs.tcsl_encode(fs.w4_decode(up4)), fs.tcsl_encode(fs.w4_decode(down4))
    z = fs.spmm_lscd(down_s, torch.relu(fs.spmm_lscd(up_s, x)))
    fs.check_device_status()
    # decoded weights are rounded once (eps / 2), hidden values once (eps / 2) in each, outputs once in each
    assert (y.double() - z.double()).norm() <= 3 * torch.finfo(torch.float16).eps * y.double().norm()


@pytest.mark.parametrize("K", [40, 135, 262])
@pytest.mark.parametrize("first", [0, 1, 2, 3])
def test_rows_that_start_anywhere(K, first):
    """Views whose rows start on odd values, and their neighbours, which nothing may read into the result."""
    whole = torch.full((37, K + 8), float("nan"), device="cuda", dtype=torch.bfloat16)
    W = whole[:, first:first + K]
    W.copy_(torch.randn((37, K), device="cuda", generator=gen(K)))
    for symmetric in (True, False):
        A, B = fs.w4_encode(W, 32, symmetric), fs.w4_encode(W.contiguous(), 32, symmetric)
        assert torch.equal(A.data, B.data)
        back = fs.w4_decode(A)
        assert torch.equal(back.float(), fs.w4_decode(A, torch.float32).bfloat16().float())
        X = torch.full((20, K + 8), float("nan"), device="cuda", dtype=torch.bfloat16)
        X[:, first:first + K].copy_(torch.randn((20, K), device="cuda", generator=gen(first)))
        assert torch.equal(fs.w4_matmul(A, X[:, first:first + K]), fs.w4_matmul(A, X[:, first:first + K].clone()))
