"""A 4-bit weight as an object: what its constructor refuses, copies, files.  Without a GPU; no call reads the data."""
import copy
import dataclasses
import io
import pickle

import pytest
import torch

import unstructured_sparse_skinny_b200 as fs
from unstructured_sparse_skinny_b200.build import build_library


@pytest.fixture(scope="module", autouse=True)
def library():
    build_library()


def data(M=200, K=300, group=64, symmetric=False, count=1):
    record = 1024 + (128 // group) * (32 if symmetric else 48)
    return torch.arange(count * -(-M // 128) * -(-K // 128) * 8 * record).to(torch.uint8).view(
        count, -(-M // 128), -(-K // 128), 8, record)


def weight(**kw):
    return fs.W4(**{**dict(data=data(), dtype=torch.float16, M=200, K=300, group=64, symmetric=False), **kw})


def same(a, b):
    return torch.equal(a.data, b.data) and all(getattr(a, n) == getattr(b, n)
                                               for n in ("dtype", "M", "K", "group", "symmetric", "stacked", "count"))


@pytest.mark.parametrize("kw", [
    dict(data=torch.zeros((1, 1, 1, 1, 1), dtype=torch.uint8)), dict(data=torch.zeros(1, dtype=torch.uint8)),
    dict(data=torch.zeros((), dtype=torch.uint8)), dict(M=4096, K=4096), dict(M=257), dict(K=385), dict(M=-1),
    dict(M=128), dict(group=32), dict(group=128), dict(group=0), dict(symmetric=True), dict(M=1 << 31),
    dict(data=data()[:, :, :, :, :-1]), dict(data=data().flatten()), dict(data=data()[:0]),
    dict(data=torch.cat([data().flatten(), data().flatten()])[8:8 + data().numel()].view(data().shape)),
    dict(data=data(count=2)),  # a stack that does not say so
    dict(data=data().transpose(3, 4).contiguous().transpose(3, 4)),
])
def test_constructor_refuses_what_the_kernels_would_read_past(kw):
    with pytest.raises((ValueError, OverflowError)) as e:
        weight(**kw)
    assert e.type is ValueError


@pytest.mark.parametrize("kw", [dict(data=data().to(torch.int8)), dict(data=data().tolist()), dict(dtype=torch.float32),
                                dict(dtype="float16"), dict(data=data().to("meta"))])
def test_constructor_refuses_types(kw):
    with pytest.raises(TypeError):
        weight(**kw)


@pytest.mark.parametrize("a", [lambda: weight(), lambda: weight(data=data(count=3), stacked=True),
                               lambda: weight(data=data(symmetric=True), symmetric=True, dtype=torch.bfloat16)])
def test_copies_and_files(a):
    a = a()
    file = io.BytesIO()
    torch.save({"layer": a}, file)
    file.seek(0)
    copies = [copy.deepcopy(a), pickle.loads(pickle.dumps(a)), torch.load(file, weights_only=False)["layer"]]
    for b in copies + [copy.copy(a), dataclasses.replace(a), dataclasses.replace(a, data=a.data.clone())]:
        assert same(a, b)
        assert b._ref._obj.data == b.data.data_ptr() and b._ref._obj is not a._ref._obj
    for b in copies:  # with data of its own
        assert b.data.data_ptr() != a.data.data_ptr()
    assert "_ref" not in repr(a)


def test_a_matrix_of_a_stack():
    a = weight(data=data(count=3), stacked=True)
    one = a.matrix(2)
    assert one.count == 1 and not one.stacked and torch.equal(one.data[0], a.data[2])
    assert one._ref._obj.data == a.data[2].data_ptr()


def test_weights_in_host_memory_are_held_but_not_multiplied():
    a, stack = weight(), weight(data=data(M=300, K=300), M=300, stacked=True)
    x = torch.zeros((2, 300), dtype=torch.float16)
    for call in (lambda: fs.w4_matmul(a, x), lambda: fs.w4_decode(a), lambda: fs.w4_matmul(a, x, stream=0),
                 lambda: fs.moe_w4(x, torch.zeros((1, 300)), stack, stack, stack, 1)):
        with pytest.raises(TypeError):
            call()
