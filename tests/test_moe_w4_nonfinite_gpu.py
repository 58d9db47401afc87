"""A non-finite weight of one expert stays with the tokens that chose the expert."""
import pytest
import torch

import unstructured_sparse_skinny_b200 as fs
from tests.test_w4_gpu import TYPES, codes_of, gen

pytestmark = pytest.mark.gpu


def stacks(E, H, F, group, dtype):
    return [codes_of(s, group, dtype, False, i) for i, s in enumerate(((E, F, H), (E, F, H), (E, H, F)))]


@pytest.mark.parametrize("T", [2, 8, 9, 20, 64])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("group", [32, 128])
def test_bad_scale_reaches_only_its_tokens(T, bad, which, group):
    """Which: of gate, up or down.  Expert 3 has one bad group; the first token takes it, the last takes none, the others take others."""
    E, H, F = 5, 264, 200
    plain = stacks(E, H, F, group, torch.bfloat16)
    X = torch.randn((T, H), device="cuda", generator=gen(T)).bfloat16()
    ids = torch.tensor([[0, 2], [4, 1], [2, 4]], device="cuda", dtype=torch.int32).repeat(22, 1)[:T].clone()
    ids[0, 1] = 3
    ids[T - 1] = -1
    weights = torch.rand((T, 2), device="cuda", generator=gen(1)) + 0.1
    clean = fs.moe_w4_experts(X, ids, weights, *(fs.w4_pack(*s, group=group) for s in plain))
    plain[which][1][3, 17, 1] = bad
    got = fs.moe_w4_experts(X, ids, weights, *(fs.w4_pack(*s, group=group) for s in plain))
    assert torch.equal(got[1:], clean[1:])
    assert (got[T - 1] == 0).all()
    if which == 2:  # row 17 of the output
        assert not torch.isfinite(got[0, 17])
        clean[0, 17] = got[0, 17] = 0
        assert torch.equal(got[0], clean[0])
    else:           # row 17 of h, which every output reads
        assert not torch.isfinite(got[0]).any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [3, 12])
def test_an_encoded_expert_with_a_nan(dtype, T):
    """As a damaged checkpoint brings it: the encoder keeps the NaN's group not finite, the layer keeps it to its tokens."""
    E, H, F, k = 4, 128, 136, 1
    g = gen(5)
    dense = [torch.randn(s, device="cuda", generator=g).mul(0.1).to(dtype) for s in ((E, F, H), (E, F, H), (E, H, F))]
    router = torch.zeros((E, H), device="cuda", dtype=dtype)
    router[torch.arange(E), torch.arange(E)] = 1
    X = torch.randn((T, H), device="cuda", generator=g).to(dtype) * 0.1
    X[torch.arange(T), torch.arange(T) % 3] = 9  # token t chooses expert t % 3
    clean = fs.moe_w4(X, router, *(fs.w4_encode(w) for w in dense), k)
    assert clean[1].flatten().tolist() == [t % 3 for t in range(T)]
    dense[2][2, 5, 7] = float("nan")
    out, _, _ = fs.moe_w4(X, router, *(fs.w4_encode(w) for w in dense), k)
    took = clean[1].flatten() == 2
    assert torch.equal(out[~took], clean[0][~took])
    assert not torch.isfinite(out[took][:, 5]).any()
