"""Router logits that are nearly equal are ordered as in exact arithmetic."""
import math

import pytest
import torch

import unstructured_sparse_skinny_b200 as fs
from tests.test_w4_gpu import TYPES, codes_of, gen

pytestmark = pytest.mark.gpu


def near_ties(E, H, dtype, relative, seed):
    """One token and an fp32 router whose odd rows' logits are their even neighbours' times 1 + relative.

    The last three columns of an odd row, with activations 1, 2^-20 and 2^-40, are set to what is missing."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(H, generator=g).to(dtype)
    x[-3:] = torch.tensor([1.0, 2.0 ** -20, 2.0 ** -40]).to(dtype) if dtype is torch.bfloat16 else \
        torch.tensor([1.0, 2.0 ** -10, 2.0 ** -20]).to(dtype)
    router = torch.randn((E, H), generator=g)
    router[:, -3:] = 0
    xs = x.double().tolist()

    def logit(row):  # products of 24 and 11 bits are exact in fp64, and fsum rounds once
        return math.fsum(w * v for w, v in zip(row.double().tolist(), xs))

    for e in range(0, E, 2):
        router[e] = torch.where(router[e] * x.float() < 0, -router[e], router[e])  # no cancellation: the logit is large
        want = logit(router[e]) * (1 + relative)
        router[e + 1] = torch.where(router[e + 1] * x.float() < 0, -router[e + 1], router[e + 1])
        for c in (H - 3, H - 2, H - 1):
            products = [w * v for w, v in zip(router[e + 1].double().tolist(), xs)]
            router[e + 1, c] = math.fsum([want] + [-p for p in products]) / xs[c]
        step = logit(router[e + 1]) - logit(router[e])
        assert 0.9 * relative < step / want < 1.1 * relative
    return x.unsqueeze(0), router


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bits", [30, 33, 36])
@pytest.mark.parametrize("E,H,T", [(32, 256, 1), (32, 1024, 2), (64, 1032, 40), (128, 2048, 1), (16, 8192, 33)])
def test_order_of_near_ties(E, H, T, bits, dtype):
    """A sum of n products is off by some n 2^-48 of it at most, and a lane adds a few dozen: 2^-36 is well apart."""
    x, router = near_ties(E, H, dtype, 2.0 ** -bits, H + bits)
    packed = [fs.w4_pack(*codes_of(s, 128, dtype, True, 1)) for s in ((E, 16, H), (E, 16, H), (E, H, 16))]
    X = x.repeat(T, 1).cuda()
    xs = x[0].double().tolist()
    exact = [math.fsum(w * v for w, v in zip(r, xs)) for r in router.double().tolist()]
    k = min(16, E)
    order = sorted(range(E), key=lambda e: (-exact[e], e))[:k]
    _, ids, _ = fs.moe_w4(X, router.cuda(), *packed, k)
    assert ids.tolist() == [order] * T
