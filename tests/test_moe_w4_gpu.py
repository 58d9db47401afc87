"""The 4-bit mixture-of-experts layer against a plain fp64 form.

Bound of one output, counted from the roundings: sums as in test_w4_gpu.py
(d = (K / 16 + 64) * 2^-23 of the sum of magnitudes), the activation's slope of
at most 1.13 and its own error of at most 2^-20, h rounded to 16 bits (eps / 2; it is kept better), the
weights' error of at most 2^-20, and the output's rounding (eps / 2).
"""
import pytest
import torch

import unstructured_sparse_skinny_b200 as fs
from tests.test_w4_gpu import TYPES, codes_of, dense64, gen

pytestmark = pytest.mark.gpu


def act64(name, g):
    if name == "silu":
        return g * torch.sigmoid(g)
    if name == "gelu":
        return 0.5 * g * (1 + torch.erf(g / 2 ** 0.5))
    return g.clamp(min=0)


def layer(E, H, F, group, dtype, symmetric=False, seed=0, up=True, whole=False):
    """Plain fp64 stacks and their packed forms."""
    dense, packed = [], []
    for i, shape in enumerate(((E, F, H), (E, F, H), (E, H, F))):
        codes, scales, zeros = codes_of(shape, group, dtype, symmetric or i == 2, seed + i, whole)
        dense.append(dense64(codes, scales, zeros, group))
        packed.append(fs.w4_pack(codes, scales, zeros, group=group))
    if not up:
        dense[1] = packed[1] = None
    return dense, packed


def route64(X, router, k, renormalize):
    logits = X.double() @ router.double().t()
    values, order = logits.sort(dim=1, descending=True, stable=True)
    e = (values - values[:, :1]).exp()
    return order[:, :k], e[:, :k] / (e[:, :k] if renormalize else e).sum(1, keepdim=True)


def experts64(X, ids, weights, dense, act, dtype):
    """(out, bound)"""
    gate, up, down = dense
    E, F, H = gate.shape
    eps, x = torch.finfo(dtype).eps, X.double()
    out, bound = torch.zeros((X.shape[0], H), dtype=torch.float64, device="cuda"), None
    bound = torch.zeros_like(out)
    for t in range(X.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            p = weights[t, j].double()
            dg = (H / 16 + 64) * 2.0 ** -23 * (gate[e].abs() @ x[t].abs())
            g = gate[e] @ x[t]
            a = act64(act, g)
            da = 1.13 * dg + 2.0 ** -20 * a.abs()
            if up is None:
                h, dh = a, da
            else:
                u = up[e] @ x[t]
                du = (H / 16 + 64) * 2.0 ** -23 * (up[e].abs() @ x[t].abs())
                h, dh = a * u, da * u.abs() + a.abs() * du + da * du
            dh = dh + eps / 2 * (h.abs() + dh)
            y, dy = down[e] @ h, down[e].abs() @ dh
            dy = dy + (F / 16 + 64) * 2.0 ** -23 * (down[e].abs() @ (h.abs() + dh))
            out[t] += p * y
            bound[t] += p.abs() * (dy + 2.0 ** -20 * (down[e].abs() @ h.abs()))
    return out, bound + eps / 2 * (out.abs() + bound) + torch.finfo(dtype).smallest_normal * eps


def check(got, want, bound, what=""):
    off = (got.double() - want).abs()
    assert (off <= bound).all(), f"{what}: {(off / bound).max().item():.3g} of the bound"


@pytest.mark.parametrize("T,E,k,H,F", [(1, 4, 1, 128, 128), (1, 8, 2, 264, 200), (3, 5, 5, 130, 77), (8, 16, 4, 256, 136),
                                       (9, 3, 2, 512, 40), (17, 8, 2, 200, 264), (40, 12, 3, 136, 128),
                                       (64, 2, 1, 128, 72), (64, 40, 8, 96, 64), (2, 512, 16, 64, 32),
                                       (8, 16, 16, 128, 136), (33, 3, 3, 640, 520), (64, 4, 4, 1024, 264)])
@pytest.mark.parametrize("dtype", TYPES)
def test_layer(T, E, k, H, F, dtype):
    group = (32, 64, 128)[(T + k) % 3]
    act = ("silu", "gelu", "relu")[(E + k) % 3]
    renormalize = T % 2 == 1
    dense, packed = layer(E, H, F, group, dtype, seed=T)
    X = torch.randn((T, H), device="cuda", generator=gen(T)).to(dtype)
    router = (torch.randn((E, H), device="cuda", generator=gen(E)) * H ** -0.5).to(dtype)
    out, ids, weights = fs.moe_w4(X, router, *packed, k, renormalize=renormalize, activation=act)
    want_ids, want_weights = route64(X, router, k, renormalize)
    assert torch.equal(ids.long(), want_ids) and ids.dtype == torch.int32
    assert torch.allclose(weights.double(), want_weights, rtol=2e-6, atol=0)
    check(out, *experts64(X, ids, weights, dense, act, dtype))
    again = fs.moe_w4_experts(X, ids, weights, *packed, activation=act)
    assert torch.equal(again, out)


@pytest.mark.parametrize("T,H,F,group,dtype", [(8, 6152, 2100, 32, torch.bfloat16), (8, 4096, 4104, 128, torch.float16),
                                               (16, 4360, 2568, 64, torch.float16), (13, 2568, 6280, 32, torch.bfloat16),
                                               (33, 5000, 1208, 128, torch.bfloat16)])
def test_long_rows(T, H, F, group, dtype):
    """Activations that shared memory holds in several parts, and a second pass over an expert's records."""
    dense, packed = layer(2, H, F, group, dtype, seed=T)
    X = torch.randn((T, H), device="cuda", generator=gen(T)).to(dtype)
    ids = torch.tensor([0, 1], device="cuda", dtype=torch.int32).repeat(T, 1)
    weights = torch.rand((T, 2), device="cuda", generator=gen(1))
    out = fs.moe_w4_experts(X, ids, weights, *packed)
    check(out, *experts64(X, ids, weights, dense, "silu", dtype))


@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("T", [1, 7, 64])
@pytest.mark.parametrize("dtype", TYPES)
def test_whole_numbers_are_exact(up, T, dtype):
    """One-hot activations, scales 1, relu: h is a whole number of at most 49 and every sum is exact."""
    E, H, F, k = 6, 256, 200, 3
    stacks = [codes_of(s, 128, dtype, True, i, True) for i, s in enumerate(((E, F, H), (E, F, H), (E, H, F)))]
    for codes, scales, _ in stacks:
        codes.clamp_(min=1)
        scales.fill_(1)
    dense = [dense64(*s, 128) for s in stacks]
    packed = [fs.w4_pack(*s) for s in stacks]
    g = gen(T)
    X = torch.zeros((T, H), device="cuda", dtype=dtype)
    X[torch.arange(T), torch.randint(0, H, (T, ), device="cuda", generator=g)] = 1
    ids = torch.stack([torch.randperm(E, device="cuda", generator=g)[:k] for _ in range(T)]).int()
    weights = torch.exp2(torch.randint(-3, 2, (T, k), device="cuda", generator=g).float())
    got = fs.moe_w4_experts(X, ids, weights, packed[0], packed[1] if up else None, packed[2], activation="relu")
    if not up:
        dense[1] = None
    want, _ = experts64(X, ids, weights, dense, "relu", dtype)
    assert torch.equal(got, want.to(dtype))


@pytest.mark.parametrize("rtype", ["own", "fp32"])
@pytest.mark.parametrize("H", [256, 131])
def test_router_types_and_ties(rtype, H):
    E, T, k = 24, 10, 6
    _, packed = layer(E, H, 64, 64, torch.bfloat16)
    X = torch.randn((T, H), device="cuda", generator=gen(1)).bfloat16()
    router = torch.randn((E, H), device="cuda", generator=gen(2)) * 0.1
    router = router if rtype == "fp32" else router.bfloat16()
    router[7] = router[3]
    router[20] = router[3]  # equal rows: the lower index first
    _, ids, weights = fs.moe_w4(X, router, *packed, k, renormalize=False)
    want_ids, want_weights = route64(X, router, k, False)
    assert torch.equal(ids.long(), want_ids)
    assert torch.allclose(weights.double(), want_weights, rtol=2e-6, atol=0)
    same = torch.zeros_like(router)
    _, ids, weights = fs.moe_w4(X, same, *packed, k)
    assert (ids == torch.arange(k, device="cuda", dtype=torch.int32)).all()
    assert torch.allclose(weights, torch.full_like(weights, 1 / k))


def test_far_logits_and_non_finite_tokens():
    E, H, T, k = 8, 128, 4, 3
    dense, packed = layer(E, H, 64, 64, torch.float16)
    router = torch.randn((E, H), device="cuda", generator=gen(2)).half()
    X = torch.randn((T, H), device="cuda", generator=gen(1)).half()
    X[1] *= 500  # logits of thousands: the softmax must not overflow
    clean = fs.moe_w4(X, router, *packed, k)
    assert torch.isfinite(clean[2]).all()
    # h is rounded to fp16 between the products: token 1's passes 65504 (computed here), the others' do not
    for t in range(T):
        h = [act64("silu", dense[0][e] @ X[t].double()) * (dense[1][e] @ X[t].double()) for e in clean[1][t].tolist()]
        fits = max(v.abs().max().item() for v in h) < 65504
        assert fits == (t != 1)
        assert torch.isfinite(clean[0][t]).all() or not fits
    X[2, 5] = float("nan")
    out, ids, weights = fs.moe_w4(X, router, *packed, k)
    assert torch.isnan(out[2]).all() and torch.isnan(weights[2]).all()
    assert (ids >= 0).all() and (ids < E).all() and len(set(ids[2].tolist())) == k
    for t in (0, 3):
        assert all(torch.equal(a[t], b[t]) for a, b in zip((out, ids, weights), clean))
    X[2, 5] = float("inf")
    out, ids, _ = fs.moe_w4(X, router, *packed, k)
    assert not torch.isfinite(out[2]).any() and len(set(ids[2].tolist())) == k
    for t in (0, 3):
        assert torch.equal(out[t], clean[0][t])


def test_ids_outside_and_twice():
    E, H, F, T = 5, 128, 72, 6
    dense, packed = layer(E, H, F, 32, torch.bfloat16)
    X = torch.randn((T, H), device="cuda", generator=gen(1)).bfloat16()
    ids = torch.tensor([[0, 0, 0], [-1, -1, -1], [2, -5, 2], [5, 1, 1 << 30], [4, 3, 2], [-1, 7, 0]], device="cuda",
                       dtype=torch.int32)
    weights = torch.rand((T, 3), device="cuda", generator=gen(3))
    weights[1] = float("nan")  # of no expert: never read into a result
    out = torch.full((T, H), 9.0, device="cuda", dtype=torch.bfloat16)
    assert fs.moe_w4_experts(X, ids, weights, *packed, out=out) is out
    want, bound = experts64(X, ids, weights, dense, "silu", torch.bfloat16)
    check(out, want, bound)
    assert (out[1] == 0).all()
    nobody = fs.moe_w4_experts(X, torch.full_like(ids, -1), weights, *packed)
    assert (nobody == 0).all()


def test_all_tokens_on_one_expert():
    dense, packed = layer(3, 256, 136, 128, torch.float16)
    X = torch.randn((64, 256), device="cuda", generator=gen(1)).half()
    ids = torch.full((64, 1), 2, device="cuda", dtype=torch.int32)
    weights = torch.ones((64, 1), device="cuda")
    check(fs.moe_w4_experts(X, ids, weights, *packed), *experts64(X, ids, weights, dense, "silu", torch.float16))


def test_strides_and_alignment():
    E, H, F, T, k = 6, 136, 64, 5, 2
    _, packed = layer(E, H, F, 64, torch.float16)
    router = torch.randn((E, H), device="cuda", generator=gen(2)).half()
    X = torch.randn((T, H), device="cuda", generator=gen(1)).half()
    want = fs.moe_w4(X, router, *packed, k)
    big = torch.full((T, H + 13), float("nan"), device="cuda", dtype=torch.float16)
    for shift in (0, 8, 5):
        big[:, shift: shift + H] = X
        got = fs.moe_w4(big[:, shift: shift + H], router, *packed, k)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    flat = torch.empty(E * H + 1, device="cuda", dtype=torch.float16)
    flat[1:].view(E, H).copy_(router)
    got = fs.moe_w4(X, flat[1:].view(E, H), *packed, k)  # a router off 16 bytes
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = torch.full((T, H + 6), 3.0, device="cuda", dtype=torch.float16)
    fs.moe_w4(X, router, *packed, k, out=out[:, 2: 2 + H])
    assert torch.equal(out[:, 2: 2 + H], want[0]) and (out[:, :2] == 3).all() and (out[:, 2 + H:] == 3).all()


def test_refusals():
    E, H, F = 4, 128, 64
    _, packed = layer(E, H, F, 64, torch.float16)
    X = torch.ones((2, H), device="cuda", dtype=torch.float16)
    router = torch.ones((E, H), device="cuda", dtype=torch.float16)
    ids, weights = torch.zeros((2, 1), device="cuda", dtype=torch.int32), torch.ones((2, 1), device="cuda")
    for bad in (lambda: fs.moe_w4(X.bfloat16(), router, *packed, 1), lambda: fs.moe_w4(X, router[:2], *packed, 1),
                lambda: fs.moe_w4(X, router.bfloat16(), *packed, 1),
                lambda: fs.moe_w4_experts(X, ids.long(), weights, *packed),
                lambda: fs.moe_w4_experts(X, ids, weights.half(), *packed)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: fs.moe_w4(X[:, :64], router, *packed, 1),
                lambda: fs.moe_w4(X, router, *packed, 1, activation="tanh"),
                lambda: fs.moe_w4_experts(X, ids[:1], weights, *packed),
                lambda: fs.moe_w4(X, router, *packed, 1, out=torch.empty_like(X[:1]))):
        with pytest.raises(ValueError):
            bad()
    for bad, status in ((lambda: fs.moe_w4(X, router, *packed, 5), 1),
                        (lambda: fs.moe_w4(X.expand(65, H) if False else X[:1].repeat(65, 1), router, *packed, 1), 2),
                        (lambda: fs.moe_w4(X, router, packed[0], packed[2], packed[2], 1), 1)):
        with pytest.raises(fs.FlashSpmmError) as e:
            bad()
        assert e.value.status == status
    assert fs.moe_w4(X[:0], router, *packed, 1)[0].shape == (0, H)


def test_workspace_is_checked():
    from unstructured_sparse_skinny_b200 import binding
    lib = binding.load_library()
    E, H, F, T = 4, 128, 64, 3
    _, (gate, up, down) = layer(E, H, F, 64, torch.float16)
    X = torch.ones((T, H), device="cuda", dtype=torch.float16)
    ids, weights = torch.zeros((T, 1), device="cuda", dtype=torch.int32), torch.ones((T, 1), device="cuda")
    out = torch.full((T, H), 5.0, device="cuda", dtype=torch.float16)
    need = lib.flashspmm_moe_w4_workspace_bytes(gate._ref, X.data_ptr(), H, T, 1)
    ws = torch.empty(need + 16, device="cuda", dtype=torch.uint8)

    def call(ptr, size):
        return lib.flashspmm_moe_w4(gate._ref, up._ref, down._ref, X.data_ptr(), H, None, 0, T, 1, 1, 0, ids.data_ptr(),
                                    weights.data_ptr(), out.data_ptr(), H, ptr, size,
                                    torch.cuda.current_stream().cuda_stream)

    assert call(None, need) == 4 and call(ws.data_ptr(), need - 1) == 4 and call(ws.data_ptr() + 8, need) == 3
    torch.cuda.synchronize()
    assert (out == 5).all()
    assert call(ws.data_ptr(), need) == 0
    assert torch.equal(out, fs.moe_w4_experts(X, ids, weights, gate, up, down))


@pytest.mark.parametrize("T,E,k,H", [(64, 128, 8, 640), (33, 300, 4, 1024), (5, 64, 3, 8192), (8, 130, 6, 2056)])
def test_wide_routing(T, E, k, H):
    """Logits by their own kernel and by the routing cluster, at sizes that split over warps and CTAs."""
    _, packed = layer(E, H, 16, 128, torch.bfloat16, symmetric=True)
    X = torch.randn((T, H), device="cuda", generator=gen(1)).bfloat16()
    router = torch.randn((E, H), device="cuda", generator=gen(2)) * H ** -0.5
    for r in (router, router.bfloat16()):
        for renormalize in (True, False):
            _, ids, weights = fs.moe_w4(X, r, *packed, k, renormalize=renormalize)
            want_ids, want_weights = route64(X, r, k, renormalize)
            assert torch.equal(ids.long(), want_ids)
            assert torch.allclose(weights.double(), want_weights, rtol=2e-6, atol=0)


@pytest.mark.parametrize("T", [1, 20])
def test_streams_and_graphs(T):
    E, H, F, k = 16, 515, 264, 4
    _, packed = layer(E, H, F, 64, torch.bfloat16)
    router = torch.randn((E, H), device="cuda", generator=gen(2)).bfloat16()
    Xs = [torch.randn((T, H), device="cuda", generator=gen(10 + i)).bfloat16() for i in range(4)]
    want = [fs.moe_w4(x, router, *packed, k) for x in Xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [fs.moe_w4(Xs[i % 4], router, *packed, k, stream=streams[i % 2]) for i in range(12)]
    torch.cuda.synchronize()
    for i in range(12):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i % 4]))
    inputs, graphs, outs = [x.clone() for x in Xs[:2]], [], []
    for x in inputs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fs.moe_w4(x, router, *packed, k))
        graphs.append(g)
    for i in (1, 3):
        inputs[0].copy_(Xs[i])
        inputs[1].copy_(Xs[i - 1])
        graphs[0].replay()
        eager = fs.moe_w4(Xs[2], router, *packed, k)
        graphs[1].replay()
        torch.cuda.synchronize()
        for a, b in ((outs[0], want[i]), (outs[1], want[i - 1]), (eager, want[2])):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_layer_from_dense_weights():
    """As a program uses it: encode the experts once, run tokens one by one and as a batch."""
    E, H, F, k, T = 8, 512, 384, 2, 6
    g = gen(1)
    gate, up = ((torch.randn((E, F, H), device="cuda", generator=g) * 0.04).bfloat16() for _ in range(2))
    down = (torch.randn((E, H, F), device="cuda", generator=g) * 0.04).bfloat16()
    packed = [fs.w4_encode(w, group=64, symmetric=False) for w in (gate, up, down)]
    dense = [fs.w4_decode(w, torch.float32).double() for w in packed]
    router = torch.randn((E, H), device="cuda", generator=g) * H ** -0.5
    X = torch.randn((T, H), device="cuda", generator=g).bfloat16()
    out, ids, weights = fs.moe_w4(X, router, *packed, k)
    check(out, *experts64(X, ids, weights, dense, "silu", torch.bfloat16))
    for t in range(T):
        one = fs.moe_w4(X[t: t + 1], router, *packed, k)
        assert torch.equal(one[1][0], ids[t])
        check(one[0], *(v[t: t + 1] for v in experts64(X, ids, weights, dense, "silu", torch.bfloat16)))
