"""4-bit weights without a GPU: buffer sizes, and every refusal that the host
makes before it touches a device (pointers below are never dereferenced)."""
import ctypes

import pytest
import torch

import unstructured_sparse_skinny_b200 as fs
from unstructured_sparse_skinny_b200 import binding
from unstructured_sparse_skinny_b200.build import build_library
from unstructured_sparse_skinny_b200.w4 import _W4View

FAKE = 0x7F0000000000
INVALID, UNSUPPORTED, ALIGNMENT, CAPACITY, NO_DEVICE = 1, 2, 3, 4, 8
F16, BF16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    build_library()
    return binding.load_library()


def view(**kw):
    v = dict(M=128, K=256, count=1, group=128, dtype=F16, zeros=0, data=FAKE)
    v.update(kw)
    return _W4View(**v)


@pytest.mark.parametrize("zeros", [0, 1])
@pytest.mark.parametrize("M,K,count,group,records", [
    (16, 128, 1, 128, 8), (129, 129, 1, 64, 32), (1, 1, 3, 32, 24), (0, 128, 1, 128, 0),
    (4099, 5003, 2, 32, 2 * 33 * 8 * 40), (1 << 20, 1 << 20, 4, 128, 4 * (1 << 16) * (1 << 13)),
])
def test_bytes(lib, M, K, count, group, records, zeros):
    groups = 16 * (128 // group)
    assert lib.flashspmm_w4_bytes(M, K, count, group, zeros) == records * (1024 + groups * (3 if zeros else 2))


@pytest.mark.parametrize("args", [(-1, 8, 1, 128, 0), (8, -1, 1, 128, 0), (8, 8, 0, 128, 0), (8, 8, 1, 16, 0),
                                  (8, 8, 1, 0, 0), (8, 8, 1, 256, 0), ((1 << 30) + 1, 8, 1, 128, 0),
                                  (8, 8, 1, 128, 2), (8, 8, 1, 128, -1)])
def test_bytes_rejects(lib, args):
    assert lib.flashspmm_w4_bytes(*args) == -1


BAD_VIEWS = [(dict(M=-1), INVALID), (dict(count=0), INVALID), (dict(group=96), UNSUPPORTED),
             (dict(dtype=F32), UNSUPPORTED), (dict(zeros=2), INVALID), (dict(data=None), INVALID),
             (dict(data=FAKE + 8), ALIGNMENT), (dict(K=(1 << 30) + 128), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", BAD_VIEWS)
def test_every_call_rejects_a_bad_view(lib, kw, status):
    v = ctypes.byref(view(**kw))
    good = ctypes.byref(view())
    assert lib.flashspmm_w4_encode(FAKE, 1 << 40, 1, v, None) == status
    assert lib.flashspmm_w4_pack(FAKE, FAKE, None, v, None) == status
    assert lib.flashspmm_w4_decode(v, FAKE, F16, None) == status
    assert lib.flashspmm_w4_matmul(v, FAKE, 1 << 40, FAKE, 1 << 40, F16, 1, None, 0, None) == status
    for three in ((v, good, good), (good, v, good), (good, good, v)):
        assert lib.flashspmm_moe_w4(*three, FAKE, 256, None, F16, 1, 1, 1, 0, FAKE, FAKE, FAKE, 256, FAKE, 1 << 30,
                                    None) == status


def test_null_view(lib):
    assert lib.flashspmm_w4_decode(None, FAKE, F16, None) == INVALID
    assert lib.flashspmm_w4_matmul(None, FAKE, 256, FAKE, 128, F16, 1, None, 0, None) == INVALID


@pytest.mark.parametrize("W,ldw,symmetric,zeros,status", [
    (FAKE, 255, 1, 0, INVALID),        # rows overlap
    (FAKE, 256, 1, 1, INVALID),        # symmetric with zero points
    (FAKE, 256, 0, 0, INVALID),        # asymmetric without
    (None, 256, 1, 0, INVALID),
    (FAKE + 1, 256, 1, 0, ALIGNMENT),
])
def test_encode_rejects(lib, W, ldw, symmetric, zeros, status):
    assert lib.flashspmm_w4_encode(W, ldw, symmetric, ctypes.byref(view(zeros=zeros)), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(N=257), UNSUPPORTED), (dict(N=-1), INVALID), (dict(ldb=255), INVALID), (dict(ldc=127), INVALID),
    (dict(c_dtype=BF16), UNSUPPORTED), (dict(c_dtype=7), UNSUPPORTED), (dict(C=None), INVALID),
    (dict(C=FAKE + 1), ALIGNMENT), (dict(C=FAKE + 2, c_dtype=F32), ALIGNMENT),
])
def test_matmul_rejects(lib, kw, status):
    a = dict(N=4, ldb=256, ldc=128, c_dtype=F16, C=FAKE)
    a.update(kw)
    rc = lib.flashspmm_w4_matmul(ctypes.byref(view()), FAKE, a["ldb"], a["C"], a["ldc"], a["c_dtype"], a["N"], None, 0,
                                 None)
    assert rc == status


def test_matmul_rejects_a_stack(lib):
    rc = lib.flashspmm_w4_matmul(ctypes.byref(view(count=2)), FAKE, 256, FAKE, 128, F16, 4, None, 0, None)
    assert rc == INVALID


def moe(lib, gate=None, up=None, down=None, **kw):
    a = dict(X=FAKE, ldx=256, router=FAKE, router_dtype=F16, tokens=4, top_k=2, activation=0, ids=FAKE, weights=FAKE,
             out=FAKE, ldo=256, workspace=FAKE, size=1 << 30)
    a.update(kw)
    g = view(count=8, **(gate or {}))
    u = view(count=8, **(up or {}))
    d = view(**{**dict(count=8, M=256, K=128), **(down or {})})
    return lib.flashspmm_moe_w4(ctypes.byref(g), ctypes.byref(u), ctypes.byref(d), a["X"], a["ldx"], a["router"],
                                a["router_dtype"], a["tokens"], a["top_k"], 1, a["activation"], a["ids"], a["weights"],
                                a["out"], a["ldo"], a["workspace"], a["size"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(down=dict(M=128)), INVALID), (dict(down=dict(K=256)), INVALID), (dict(down=dict(count=7)), INVALID),
    (dict(down=dict(group=64)), INVALID), (dict(down=dict(dtype=BF16)), INVALID), (dict(up=dict(M=112)), INVALID),
    (dict(up=dict(dtype=BF16)), INVALID), (dict(tokens=65), UNSUPPORTED), (dict(tokens=-1), INVALID),
    (dict(top_k=0), INVALID), (dict(top_k=9), INVALID), (dict(router=None, top_k=17), UNSUPPORTED),
    (dict(ldx=255), INVALID), (dict(ldo=255), INVALID), (dict(activation=3), UNSUPPORTED),
    (dict(router_dtype=BF16), UNSUPPORTED), (dict(X=None), INVALID), (dict(out=None), INVALID),
    (dict(ids=None), INVALID), (dict(weights=None), INVALID), (dict(X=FAKE + 1), ALIGNMENT),
    (dict(ids=FAKE + 2), ALIGNMENT), (dict(router=FAKE + 2, router_dtype=F32), ALIGNMENT),
])
def test_moe_rejects(lib, kw, status):
    assert moe(lib, **kw) == status


def test_moe_rejects_too_many_experts(lib):
    g, d = view(count=513), view(count=513, M=256, K=128)
    rc = lib.flashspmm_moe_w4(ctypes.byref(g), None, ctypes.byref(d), FAKE, 256, FAKE, F16, 4, 2, 1, 0, FAKE, FAKE,
                              FAKE, 256, FAKE, 1 << 40, None)
    assert rc == UNSUPPORTED


def test_moe_without_tokens_does_nothing(lib):
    assert moe(lib, tokens=0, X=None, out=None, ids=None, weights=None, workspace=None, size=0) == 0


def test_empty_matrices_do_nothing(lib):
    for kw in (dict(M=0), dict(K=0)):
        v = ctypes.byref(view(data=None, **kw))
        assert lib.flashspmm_w4_encode(None, 256, 1, v, None) == 0
        assert lib.flashspmm_w4_pack(None, None, None, v, None) == 0
        assert lib.flashspmm_w4_decode(v, None, F16, None) == 0
    assert lib.flashspmm_w4_matmul(ctypes.byref(view(M=0)), None, 256, None, 0, F16, 4, None, 0, None) == 0
    assert lib.flashspmm_w4_matmul(ctypes.byref(view()), None, 256, None, 128, F16, 0, None, 0, None) == 0


def test_no_device_is_reported(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    v = ctypes.byref(view())
    assert lib.flashspmm_w4_encode(FAKE, 256, 1, v, None) == NO_DEVICE
    assert lib.flashspmm_w4_decode(v, FAKE, F32, None) == NO_DEVICE
    assert lib.flashspmm_w4_matmul(v, FAKE, 256, FAKE, 128, F16, 4, None, 0, None) == NO_DEVICE
    assert moe(lib) == NO_DEVICE


def test_python_calls_refuse_host_tensors():
    W = torch.zeros((16, 128), dtype=torch.float16)
    with pytest.raises(TypeError):
        fs.w4_encode(W)
    with pytest.raises(TypeError):
        fs.w4_pack(W.to(torch.uint8), W[:, :1])
