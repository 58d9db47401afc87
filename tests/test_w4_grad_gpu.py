"""Inference calls refuse tensors that autograd tracks, outputs among them, and take them without grad mode."""
import pytest
import torch

import unstructured_sparse_skinny_b200 as fs
from tests.test_w4_gpu import codes_of, gen

pytestmark = pytest.mark.gpu


def test_outputs():
    stack = [fs.w4_pack(*codes_of((2, 128, 128), 128, torch.float16, True, i)) for i in range(3)]
    A = stack[0].matrix(0)
    B = torch.randn((3, 128), device="cuda", generator=gen(1)).half()
    ids, weights = torch.zeros((3, 1), device="cuda", dtype=torch.int32), torch.ones((3, 1), device="cuda")
    out = torch.zeros((3, 128), device="cuda", dtype=torch.float16, requires_grad=True)
    for call in (lambda: fs.w4_matmul(A, B, out), lambda: fs.moe_w4_experts(B, ids, weights, *stack, out=out)):
        with pytest.raises(RuntimeError):
            call()
        assert (out == 0).all()
        with torch.no_grad():
            assert call() is out
            assert (out != 0).any()
            out.zero_()
