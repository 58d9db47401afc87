"""4-bit weights with group scales: encoder, skinny product and the
mixture-of-experts layer (argument marshalling only; see "4-bit weights" in
``include/flashspmm.h``).

A weight is ``w = s * (q - z)`` with codes q in 0..15, one scale s (float16 or
bfloat16) and, unless it is symmetric, one zero point z for each group of 32,
64 or 128 neighbours along K.  Activations have the scales' type.

Every call runs on the device of its tensors.  ``stream`` is a
``torch.cuda.Stream``, a raw handle or None for the current stream of that
device; outputs and scratch are allocated on the stream the call runs on, so
calls on different streams share nothing and every call can be captured in a
CUDA graph.  Inputs made on another stream are ordered by the caller, as with
torch's own operators.  Errors that a kernel finds are read with
``check_device_status``.  These are inference calls: an input, or an output
that the caller gives, that requires grad is refused while grad mode is on.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, fields

import torch

from . import binding

_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_ACTIVATIONS = {"silu": 0, "gelu": 1, "relu": 2}


class _W4View(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("K", ctypes.c_int32), ("count", ctypes.c_int32), ("group", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("zeros", ctypes.c_int32), ("data", ctypes.c_void_p)]


def _overlap(a: torch.Tensor, lda: int, b: torch.Tensor, ldb: int) -> bool:
    """Whether rows of a and of b (as many; their distances in values) share memory, to be safe also where only their
    ranges meet, unless equal distances keep their columns apart."""
    rows, (wa, wb) = a.shape[0], (t.shape[1] * t.element_size() for t in (a, b))
    if rows == 0 or wa == 0 or wb == 0:
        return False
    pa, pb, at, bt = lda * a.element_size(), ldb * b.element_size(), a.data_ptr(), b.data_ptr()
    if at >= bt + (rows - 1) * pb + wb or bt >= at + (rows - 1) * pa + wa:
        return False
    apart = (bt - at) % pa if pa == pb else 0
    return rows == 1 or not (wa <= apart <= pa - wb)


def _shape(count: int, M: int, K: int, group: int, symmetric: bool) -> tuple:
    """Shape of the data of ``count`` matrices."""
    nbytes = binding.load_library().flashspmm_w4_bytes(M, K, count, group, int(not symmetric))
    if nbytes < 0:
        raise ValueError(f"4-bit weights need group 32, 64 or 128 and at least one matrix, got group {group}, "
                         f"{count} of {M} x {K}")
    blocks, units = -(-M // 128), -(-K // 128)
    return count, blocks, units, 8, nbytes // max(1, count * blocks * units * 8)


@dataclass(frozen=True, eq=False)
class W4:
    """A 4-bit matrix [M, K], or a stack [count, M, K], in device memory.

    It can be copied, pickled and saved.  Data in host memory, as a file loaded
    without a GPU leaves them, can be held but not multiplied;
    ``dataclasses.replace(A, data=A.data.cuda())`` moves them."""
    data: torch.Tensor   # uint8 [count, blocks, units, 8, record]: blocks of 128 rows, units of 128 columns
    dtype: torch.dtype   # of the scales, and of the activations they meet: float16 or bfloat16
    M: int
    K: int
    group: int
    symmetric: bool      # without zero points: every one is 8
    stacked: bool = False  # made from a 3-D tensor

    def __post_init__(self):
        if not isinstance(self.data, torch.Tensor) or self.data.dtype is not torch.uint8 or \
                self.data.device.type not in ("cuda", "cpu"):
            raise TypeError("data must be a uint8 tensor")
        if self.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("dtype must be torch.float16 or torch.bfloat16")
        count = self.data.shape[0] if self.data.dim() else 0
        shape = _shape(count, self.M, self.K, self.group, self.symmetric)
        if tuple(self.data.shape) != shape or not self.data.is_contiguous() or self.data.data_ptr() % 16 != 0 or \
                (count != 1 and not self.stacked):
            raise ValueError(f"data must be a contiguous {list(shape)} tensor on a 16-byte boundary, "
                             f"got {list(self.data.shape)}")
        # the kernels' view: byref keeps the structure alive, and a copy makes its own
        v = _W4View(self.M, self.K, count, self.group, _DTYPES[self.dtype], int(not self.symmetric),
                    self.data.data_ptr() or None)
        object.__setattr__(self, "_ref", ctypes.byref(v))

    def __getstate__(self):
        return {f.name: getattr(self, f.name) for f in fields(self)}

    def __setstate__(self, state):
        for name, value in state.items():
            object.__setattr__(self, name, value)
        self.__post_init__()

    @property
    def count(self) -> int:
        return int(self.data.shape[0])

    @property
    def device(self) -> torch.device:
        return self.data.device

    @property
    def nbytes(self) -> int:
        return int(self.data.numel())

    def matrix(self, index: int) -> "W4":
        """One matrix of a stack as a view; nothing is copied."""
        if not 0 <= index < self.count:
            raise IndexError(f"matrix {index} of a stack of {self.count}")
        return W4(self.data[index:index + 1], self.dtype, self.M, self.K, self.group, self.symmetric)


class _On:
    """Makes a tensor's device and the stream that a caller named current."""

    def __init__(self, device: torch.device, stream):
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else \
                torch.cuda.default_stream(device)
        if stream is not None and stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        self._device, self._stream = torch.cuda.device(device), torch.cuda.stream(stream)

    def __enter__(self):
        self._device.__enter__()
        self._stream.__enter__()

    def __exit__(self, *exc):
        self._stream.__exit__(*exc)
        self._device.__exit__(*exc)


def _elsewhere(device: torch.device, stream) -> bool:
    if device.index is None:  # host memory
        raise TypeError(f"4-bit weights are multiplied on a GPU, these are on {device}")
    return stream is not None or torch.cuda.current_device() != device.index


def _raw_stream(device: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def _scratch(nbytes: int, like: torch.Tensor):
    return like.new_empty(nbytes, dtype=torch.uint8) if nbytes else None


def _cuda(t, name: str, dtypes) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a CUDA tensor of type " + " or ".join(str(d) for d in dtypes))


def _no_grad(*tensors) -> None:
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise RuntimeError("4-bit weights have no backward pass: call this under torch.no_grad()")


def _rows(t: torch.Tensor) -> tuple:
    """A 2-D tensor with unit stride along its rows, and the distance of its rows."""
    if t.is_contiguous():
        return t, t.shape[1]
    if t.shape[1] > 1 and t.stride(1) != 1 or t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        t = t.contiguous()
    return t, (t.stride(0) if t.shape[0] > 1 else t.shape[1])


def _output(t, shape: tuple, dtypes, device: torch.device, name: str) -> int:
    """Checks an output that the caller gave; the distance of its rows."""
    _cuda(t, name, dtypes)
    _no_grad(t)
    if t.shape != shape or t.device != device or (shape[1] > 1 and t.stride(1) != 1) or \
            (shape[0] > 1 and t.stride(0) < shape[1]):
        raise ValueError(f"{name} must be a {list(shape)} tensor on {device} with unit stride along its rows")
    return t.stride(0) if shape[0] > 1 else shape[1]


def _empty(shape, dtype: torch.dtype, group: int, symmetric: bool, device: torch.device) -> W4:
    """Unwritten data for a weight of shape [M, K] or [count, M, K]."""
    count, (M, K) = (shape[0] if len(shape) == 3 else 1), shape[-2:]
    return W4(torch.empty(_shape(count, M, K, group, symmetric), dtype=torch.uint8, device=device), dtype, M, K, group,
              symmetric, len(shape) == 3)


def w4_encode(W: torch.Tensor, group: int = 128, symmetric: bool = True, stream=None) -> W4:
    """Quantise a dense float16 or bfloat16 weight ``[M, K]`` (or a stack
    ``[count, M, K]``) on the GPU: symmetric codes around 8, or asymmetric
    ones with a zero point per group."""
    _cuda(W, "W", (torch.float16, torch.bfloat16))
    if W.dim() not in (2, 3):
        raise TypeError("W must have 2 or 3 dimensions")
    _no_grad(W)
    if _elsewhere(W.device, stream):
        with _On(W.device, stream):
            return w4_encode(W, group, symmetric)
    if W.dim() == 3:
        rows, ldw = W.contiguous(), W.shape[2]
    else:
        rows, ldw = _rows(W)
    A = _empty(W.shape, W.dtype, group, symmetric, W.device)
    binding._check(binding.load_library().flashspmm_w4_encode(rows.data_ptr() or None, ldw, int(symmetric), A._ref,
                                                              _raw_stream(W.device)), "w4_encode")
    return A


def w4_pack(codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None, group: int = 128,
            stream=None) -> W4:
    """Lay out codes quantised elsewhere: uint8 ``codes`` ``[M, K]`` (or
    ``[count, M, K]``) of 0..15, ``scales`` and uint8 ``zeros`` (0..63; None =
    all 8) of ``[M, ceil(K / group)]`` (or with count)."""
    _cuda(codes, "codes", (torch.uint8, ))
    _cuda(scales, "scales", (torch.float16, torch.bfloat16))
    if codes.dim() not in (2, 3):
        raise TypeError("codes must have 2 or 3 dimensions")
    _no_grad(scales)
    if _elsewhere(codes.device, stream):
        with _On(codes.device, stream):
            return w4_pack(codes, scales, zeros, group)
    A = _empty(codes.shape, scales.dtype, group, zeros is None, codes.device)
    per = (*codes.shape[:-1], -(-codes.shape[-1] // group))
    if zeros is not None:
        _cuda(zeros, "zeros", (torch.uint8, ))
    for name, t in (("scales", scales), ("zeros", zeros)):
        if t is not None and (t.shape != per or t.device != codes.device):
            raise ValueError(f"{name} must be a {list(per)} tensor on {codes.device}")
    codes, scales, zeros = codes.contiguous(), scales.contiguous(), None if zeros is None else zeros.contiguous()
    binding._check(binding.load_library().flashspmm_w4_pack(
        codes.data_ptr() or None, scales.data_ptr() or None, None if zeros is None else zeros.data_ptr() or None,
        A._ref, _raw_stream(codes.device)), "w4_pack")
    return A


def w4_decode(A: W4, dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """The dense weight ``s * (q - z)`` in A's type (rounded once) or, with
    ``dtype=torch.float32``, exactly."""
    dtype = A.dtype if dtype is None else dtype
    if dtype not in _DTYPES:
        raise TypeError("dtype must be the weight's own or torch.float32")
    if _elsewhere(A.device, stream):
        with _On(A.device, stream):
            return w4_decode(A, dtype)
    shape = (A.count, A.M, A.K) if A.stacked else (A.M, A.K)
    W = torch.empty(shape, dtype=dtype, device=A.device)
    binding._check(binding.load_library().flashspmm_w4_decode(A._ref, W.data_ptr() or None, _DTYPES[dtype],
                                                              _raw_stream(A.device)), "w4_decode")
    return W


def w4_matmul(A: W4, B: torch.Tensor, C: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """C = A x B for a skinny B.  B is ``[N, K]`` in A's type with N = 1..256
    (rows may be apart); returns C as ``[N, M]`` in that type, or writes the
    given C, which must not overlap B.  With a 16-bit C and N > 8 weights may be
    rounded to that type before the product; with a float32 C neither weights
    nor sums are (about twice the time for large N)."""
    lib = binding._lib or binding.load_library()
    device, dtype = A.data.device, A.dtype
    if B.dtype is not dtype or B.dim() != 2 or B.device != device:
        raise TypeError(f"B must be a 2-D {dtype} tensor on {device}")
    if _elsewhere(device, stream):
        with _On(device, stream):
            return w4_matmul(A, B, C)
    _no_grad(B)
    if B.shape[1] != A.K:
        raise ValueError(f"B has shape {tuple(B.shape)}, expected (N, {A.K})")
    B, ldb = _rows(B)
    N = B.shape[0]
    if C is None:
        C, ldc, c_type = B.new_empty((N, A.M)), A.M, _DTYPES[dtype]
    else:
        ldc, c_type = _output(C, (N, A.M), (dtype, torch.float32), device, "C"), _DTYPES[C.dtype]
        if _overlap(B, ldb, C, ldc):
            raise ValueError("C must not overlap B, which is read while C is written")
    ptr = B.data_ptr()
    need = lib.flashspmm_w4_matmul_workspace_bytes(A._ref, ptr, ldb, N)
    ws = _scratch(need, B)
    status = lib.flashspmm_w4_matmul(A._ref, ptr, ldb, C.data_ptr(), ldc, c_type, N,
                                     None if ws is None else ws.data_ptr(), need, _raw_stream(device))
    if status:
        binding._check(status, "w4_matmul")
    return C


def _moe(X, router, gate, up, down, top_k, renormalize, activation, ids, weights, out):
    lib = binding._lib or binding.load_library()
    device, dtype = gate.data.device, gate.dtype
    X, ldx = _rows(X)
    T = X.shape[0]
    if out is None:
        out, ldo = X.new_empty((T, gate.K)), gate.K
    else:
        ldo = _output(out, (T, gate.K), (dtype, ), device, "out")
    ptr = X.data_ptr()
    need = lib.flashspmm_moe_w4_workspace_bytes(gate._ref, ptr, ldx, T, top_k)
    ws = _scratch(need, X)
    status = lib.flashspmm_moe_w4(
        gate._ref, None if up is None else up._ref, down._ref, ptr, ldx, None if router is None else router.data_ptr(),
        _DTYPES[dtype if router is None else router.dtype], T, top_k, renormalize, activation, ids.data_ptr(),
        weights.data_ptr(), out.data_ptr(), ldo, None if ws is None else ws.data_ptr(), need, _raw_stream(device))
    if status:
        binding._check(status, "moe_w4")
    return out


def _check_experts(X, gate: W4, up, down: W4, activation: str) -> None:
    device, dtype = gate.data.device, gate.dtype
    if X.dtype is not dtype or X.dim() != 2 or X.device != device:
        raise TypeError(f"X must be a 2-D {dtype} tensor on {device}")
    if X.shape[1] != gate.K:
        raise ValueError(f"X has shape {tuple(X.shape)}, expected (T, {gate.K})")
    if activation not in _ACTIVATIONS:
        raise ValueError("activation must be one of " + ", ".join(_ACTIVATIONS))
    for w in (up, down):
        if w is not None and w.data.device != device:
            raise ValueError("the experts' weights must be on one device")


def moe_w4(X: torch.Tensor, router: torch.Tensor, gate: W4, up: W4 | None, down: W4, top_k: int,
           renormalize: bool = True, activation: str = "silu", out: torch.Tensor | None = None, stream=None) -> tuple:
    """A mixture-of-experts layer for T = 1..64 tokens: ``(out, ids, weights)``.

    X        ``[T, H]``;  router  ``[E, H]`` in X's type or float32.
    gate, up stacks ``[E, F, H]`` (``up=None``: no gate product);  down  ``[E, H, F]``.
    The token's ``top_k`` experts (ties to the lower index) are weighted with
    the softmax over their logits (``renormalize``) or over all logits, and
    ``out = sum weights * down(act(gate x) * up x)``.  ``activation`` is
    "silu", "gelu" (with erf) or "relu".  ``ids`` is int32 and ``weights``
    float32, both ``[T, top_k]``, the largest first."""
    _check_experts(X, gate, up, down, activation)
    device = gate.data.device
    if (router.dtype is not X.dtype and router.dtype is not torch.float32) or router.device != device or \
            router.shape != (gate.data.shape[0], gate.K):
        raise TypeError(f"router must be a [{gate.count}, {gate.K}] tensor of X's type or float32 on {device}")
    if _elsewhere(device, stream):
        with _On(device, stream):
            return moe_w4(X, router, gate, up, down, top_k, renormalize, activation, out)
    _no_grad(X, router)
    ids = X.new_empty((X.shape[0], top_k), dtype=torch.int32)
    weights = X.new_empty((X.shape[0], top_k), dtype=torch.float32)
    out = _moe(X, router.contiguous(), gate, up, down, top_k, int(renormalize), _ACTIVATIONS[activation], ids, weights,
               out)
    return out, ids, weights


def moe_w4_experts(X: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate: W4, up: W4 | None, down: W4,
                   activation: str = "silu", out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The experts of ``moe_w4`` under the caller's own routing: int32 ``ids``
    and float32 ``weights`` of ``[T, top_k]``.  An id outside 0..E-1 (padding,
    or an expert of another rank) contributes nothing; a token whose ids are
    all outside gets zeros."""
    _check_experts(X, gate, up, down, activation)
    device = gate.data.device
    _cuda(ids, "ids", (torch.int32, ))
    _cuda(weights, "weights", (torch.float32, ))
    if ids.dim() != 2 or ids.shape[0] != X.shape[0] or weights.shape != ids.shape or ids.device != device or \
            weights.device != device:
        raise ValueError(f"ids and weights must be [T, top_k] tensors on {device}")
    if _elsewhere(device, stream):
        with _On(device, stream):
            return moe_w4_experts(X, ids, weights, gate, up, down, activation, out)
    _no_grad(X, weights)
    return _moe(X, None, gate, up, down, ids.shape[1], 1, _ACTIVATIONS[activation], ids.contiguous(),
                weights.contiguous(), out)
