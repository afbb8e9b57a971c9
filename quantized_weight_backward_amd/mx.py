"""Binding of the microscaled 4-bit operators and the expert layer
(include/retro_mx.h): marshals torch tensors into the C ABI and nothing else.

    quantize            packed MXFP4 / NVFP4 blocks from floats
    mx_quantize(_both)  microscaled matrices along rows, columns, or both
    mx_from_blocks      a resident packed MXFP4 weight, laid out for the products
    mx_mul_mat          A B^T of two microscaled matrices
    mx_linear           x W^T with x quantised in the call
    mx_linear_backward  its gradients with respect to x and W
    mx_moe              a mixture-of-experts layer for a few tokens

Every call runs asynchronously on `stream` (default: torch's current stream of
the operands' device); outputs and scratch it allocates belong to that stream.
None is recorded for autograd: results require no gradient, also where an
operand does. mx_linear's gradients come from mx_linear_backward; mx_moe, for
serving, has none.
"""

from __future__ import annotations

import functools

import torch

from . import (BF16, E_SHAPE, E_TYPE, F16, F32, MXFP4, TYPES, _check, _current_device, _device_tensor, _raw_stream, lib,
               row_bytes)

_FLOAT = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
MX_VARIANT_AUTO, MX_VARIANT_SIMPLE, MX_VARIANT_TILE_256x256, MX_VARIANT_TILE_128x128, MX_VARIANT_TILE_64x128, \
    MX_VARIANT_TILE_64x64, MX_VARIANT_SKINNY, MX_VARIANT_TILE_64x64_K4, MX_VARIANT_TILE_32x64_K4, \
    MX_VARIANT_TILE_256x192 = range(10)
MX_VARIANT_NAMES = {MX_VARIANT_SIMPLE: "simple", MX_VARIANT_TILE_256x256: "tile_256x256",
                    MX_VARIANT_TILE_128x128: "tile_128x128", MX_VARIANT_TILE_64x128: "tile_64x128",
                    MX_VARIANT_TILE_64x64: "tile_64x64", MX_VARIANT_SKINNY: "skinny",
                    MX_VARIANT_TILE_64x64_K4: "tile_64x64_k4", MX_VARIANT_TILE_32x64_K4: "tile_32x64_k4",
                    MX_VARIANT_TILE_256x192: "tile_256x192"}


def _elsewhere(t, stream) -> bool:
    """Whether a call on t has to be made under another current stream or device."""
    return stream is not None or t.get_device() != _device()


def _on(t, stream):
    """t's device, and `stream` or its current stream, as torch's current ones:
    what a call allocates belongs to the stream that it runs on."""
    if stream is None:
        return torch.cuda.device(t.device)
    if stream.device != t.device:
        raise ValueError("stream must be of the operands' device")
    return torch.cuda.stream(stream)


# the current device, and its current stream's handle
if _raw_stream is not None and _current_device is not None:
    _device = _current_device

    def _handle():
        return _raw_stream(_device())
else:
    _device = torch.cuda.current_device

    def _handle():
        return torch.cuda.current_stream().cuda_stream


def _floats(t, name):
    """(type, row stride) of a 2-D float view with contiguous rows."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    code = _FLOAT.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    along_rows, along_cols = t.stride()
    if cols > 1 and along_cols != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return code, (along_rows if rows > 1 else cols)


def _one_device(a, *others):
    at = a.get_device()
    for t in others:
        if t.get_device() != at:
            raise ValueError("all operands must be on one device")


def _given(out, rows, cols, dtype, like):
    """The row stride of a caller's output."""
    ld = _floats(out, "out")[1]
    if out.dtype != dtype or out.shape[0] != rows or out.shape[1] != cols:
        raise ValueError(f"out must be {dtype} of shape {(rows, cols)}")
    _one_device(like, out)
    return ld


# sizes of shapes that come again and again
@functools.lru_cache(maxsize=1024)
def _linear_workspace(xtype: int, K: int, N: int, T: int) -> int:
    return lib.retro_mx_linear_workspace_size(xtype, K, N, T)


@functools.lru_cache(maxsize=1024)
def _moe_workspace(xtype: int, T: int, D: int, F: int, E: int, top_k: int) -> int:
    return lib.retro_moe_workspace_size(xtype, T, D, F, E, top_k)


class MXMatrix:
    """A microscaled 4-bit matrix of `rows` x K: 32 elements along K share a
    power-of-two scale.

    codes   uint8 [rows, ceil(K / 256) * 128]
    scales  uint8 [ceil(K / 256), rows, 8]

    in the layout of include/retro_mx.h (codes past K are zero).
    """

    __slots__ = ("_codes", "_scales", "_both", "K", "rows")

    def __init__(self, codes, scales, K: int):
        self._codes, self._scales, self._both, self.K, self.rows = codes, scales, None, K, None
        self._validate()

    def _validate(self):
        """Refuses given arrays that are not (or, having got other storage or
        sizes since, no longer are) a matrix of this size."""
        codes, scales, steps = self._codes, self._scales, self._steps
        _device_tensor(codes, "codes")
        _device_tensor(scales, "scales")
        shape = codes.shape
        if codes.dtype is not torch.uint8 or len(shape) != 2 or shape[1] != steps * 128:
            raise ValueError(f"codes must be uint8 [rows, {steps * 128}] for K = {self.K}")
        if self.rows is None:
            self.rows = shape[0]
        elif shape[0] != self.rows:
            raise ValueError(f"codes has {shape[0]} rows, the matrix had {self.rows}")
        if scales.dtype is not torch.uint8 or scales.shape != (steps, shape[0], 8):
            raise ValueError(f"scales must be uint8 [{steps}, {shape[0]}, 8]")
        _one_device(codes, scales)

    @classmethod
    def _new(cls, rows: int, K: int, like):
        """Both arrays in one allocation on like's device and the current stream."""
        m = cls.__new__(cls)
        m._codes = m._scales = None
        m._both = torch.empty(rows * -(-K // 256) * 136, dtype=torch.uint8, device=like.device)
        m.K, m.rows = K, rows
        return m

    def _planes(self):
        """The arrays' addresses now: a caller's tensors may get other storage
        between two calls."""
        if self._both is None:
            return self._codes.data_ptr(), self._scales.data_ptr()
        at = self._both.data_ptr()
        return at, at + self.rows * -(-self.K // 256) * 128

    # of a matrix made here, views made anew: what is done to one is not done to the matrix
    @property
    def codes(self):
        if self._both is None:
            return self._codes
        return self._both[:self.rows * self._steps * 128].view(self.rows, self._steps * 128)

    @property
    def scales(self):
        if self._both is None:
            return self._scales
        return self._both[self.rows * self._steps * 128:].view(self._steps, self.rows, 8)

    @property
    def _steps(self):
        return -(-self.K // 256)

    @property
    def shape(self):
        return self.rows, self.K

    @property
    def device(self):
        return (self._codes if self._both is None else self._both).device

    def get_device(self) -> int:
        return (self._codes if self._both is None else self._both).get_device()


def _matrix(m, name):
    if not isinstance(m, MXMatrix):
        raise ValueError(f"{name} must be an MXMatrix")
    if m._both is None:
        m._validate()


def quantize(wtype: int, x, out=None, stream=None):
    """Packed blocks (uint8 [N, row_bytes(wtype, K)]) of an N x K float tensor
    with contiguous rows, wtype MXFP4 or NVFP4."""
    xtype, ldx = _floats(x, "x")
    if _elsewhere(x, stream):
        with _on(x, stream):
            return quantize(wtype, x, out)
    N, K = x.shape
    rb = row_bytes(wtype, K)
    if rb < 0:
        _check(E_SHAPE if wtype in TYPES.values() else E_TYPE)
    if out is None:
        out = torch.empty((N, rb), dtype=torch.uint8, device=x.device)
    else:
        _device_tensor(out, "out")
        if out.dtype != torch.uint8 or out.numel() != N * rb:
            raise ValueError(f"out must hold {N * rb} bytes")
        _one_device(x, out)
    _check(lib.retro_quantize(wtype, xtype, x.data_ptr(), ldx, out.data_ptr(), K, N, _handle()))
    return out


def mx_quantize(x, axis: int = 1, stream=None) -> MXMatrix:
    """The microscaled matrix of a 2-D float tensor with contiguous rows:
    axis 1 (or -1) along its rows, axis 0 of its transpose, blocks along the
    columns."""
    if axis not in (0, 1, -1):
        raise ValueError("axis must be 0, 1 or -1")
    xtype, ldx = _floats(x, "x")
    if _elsewhere(x, stream):
        with _on(x, stream):
            return mx_quantize(x, axis)
    T, K = x.shape
    if axis == 0:
        m = MXMatrix._new(K, T, x)
        _check(lib.retro_mx_quantize(xtype, x.data_ptr(), ldx, T, K, None, None, *m._planes(), _handle()))
    else:
        m = MXMatrix._new(T, K, x)
        _check(lib.retro_mx_quantize(xtype, x.data_ptr(), ldx, T, K, *m._planes(), None, None, _handle()))
    return m


def mx_quantize_both(x, stream=None) -> tuple[MXMatrix, MXMatrix]:
    """mx_quantize along axis 1 and axis 0 from one reading of x."""
    xtype, ldx = _floats(x, "x")
    if _elsewhere(x, stream):
        with _on(x, stream):
            return mx_quantize_both(x)
    T, K = x.shape
    r, c = MXMatrix._new(T, K, x), MXMatrix._new(K, T, x)
    _check(lib.retro_mx_quantize(xtype, x.data_ptr(), ldx, T, K, *r._planes(), *c._planes(), _handle()))
    return r, c


def mx_dequantize(m: MXMatrix, dtype=torch.float32, out=None, stream=None):
    """The values of a microscaled matrix, rows x K of dtype."""
    _matrix(m, "m")
    ytype = _FLOAT.get(dtype)
    if ytype is None:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    if _elsewhere(m, stream):
        with _on(m, stream):
            return mx_dequantize(m, dtype, out)
    rows, ld = m.rows, m.K
    if out is None:
        out = torch.empty((rows, ld), dtype=dtype, device=m.device)
    else:
        ld = _given(out, rows, ld, dtype, m)
    _check(lib.retro_mx_dequantize(ytype, *m._planes(), out.data_ptr(), ld, m.K, rows, _handle()))
    return out


def mx_from_blocks(W, K: int, N: int, stream=None) -> MXMatrix:
    """The microscaled matrix of N rows of packed MXFP4 blocks (same values)."""
    _device_tensor(W, "W")
    rb = row_bytes(MXFP4, K)
    if rb < 0:
        _check(E_SHAPE)
    if W.numel() * W.element_size() != N * rb:
        raise ValueError(f"W holds {W.numel() * W.element_size()} bytes, expected N*row_bytes = {N * rb}")
    if _elsewhere(W, stream):
        with _on(W, stream):
            return mx_from_blocks(W, K, N)
    m = MXMatrix._new(N, K, W)
    _check(lib.retro_mx_from_blocks(W.data_ptr(), *m._planes(), K, N, _handle()))
    return m


def mx_mul_mat_choice(K: int, N: int, T: int, dtype=torch.float32) -> int:
    """The kernel mx_mul_mat runs for a contiguous T x N result (a key of MX_VARIANT_NAMES)."""
    ytype = _FLOAT.get(dtype)
    if ytype is None:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    return int(lib.retro_mx_mul_mat_choice(ytype, int(N), int(K), int(N), int(T)))


def mx_mul_mat(a: MXMatrix, b: MXMatrix, dtype=torch.float32, out=None, variant: int = MX_VARIANT_AUTO, stream=None):
    """Y[t][n] = sum_k a[t][k] b[n][k] (T x N of dtype)."""
    _matrix(a, "a")
    _matrix(b, "b")
    if a.K != b.K:
        raise ValueError(f"a has K = {a.K}, b has K = {b.K}")
    ytype = _FLOAT.get(dtype)
    if ytype is None:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    _one_device(a, b)
    if _elsewhere(a, stream):
        with _on(a, stream):
            return mx_mul_mat(a, b, dtype, out, variant)
    T, N = a.rows, b.rows
    if out is None:
        out, ld = torch.empty((T, N), dtype=dtype, device=a.device), N
    else:
        ld = _given(out, T, N, dtype, a)
    _check(lib.retro_mx_mul_mat_variant(variant, ytype, *a._planes(), *b._planes(), out.data_ptr(), ld, a.K, N, T,
                                        _handle()))
    return out


def mx_linear(x, w: MXMatrix, out=None, stream=None):
    """y = x w^T for x a T x K float tensor, quantised along its rows in the
    call; y has x's type."""
    xtype, ldx = _floats(x, "x")
    _matrix(w, "w")
    T, K = x.shape
    N = w.rows
    if K != w.K:
        raise ValueError(f"x has K = {K}, w has K = {w.K}")
    _one_device(x, w)
    if _elsewhere(x, stream):
        with _on(x, stream):
            return mx_linear(x, w, out)
    if out is None:
        out, ld = torch.empty((T, N), dtype=x.dtype, device=x.device), N
    else:
        ld = _given(out, T, N, x.dtype, x)
    need = _linear_workspace(xtype, K, N, T)
    ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need > 0 else None
    _check(lib.retro_mx_linear(xtype, x.data_ptr(), ldx, *w._planes(), out.data_ptr(), ld, K, N, T,
                               None if ws is None else ws.data_ptr(), need, _handle()))
    return out


def mx_linear_backward(dy, x, wt: MXMatrix, stream=None):
    """The gradients of y = x w^T taken through the 4-bit products (the
    rounding's own derivative is taken as 1):

        dx[t][k] = sum_n dy[t][n] w[n][k]      dy along n, wt = w^T along n
        dw[n][k] = sum_t dy[t][n] x[t][k]      dy^T and x^T along t

    dy is T x N, x is T x K, wt the K x N microscaled matrix of w's transpose
    (mx_quantize(w, axis=0)). dx has dy's type, dw is float32."""
    _floats(dy, "dy")
    _floats(x, "x")
    _matrix(wt, "wt")
    T, N = dy.shape
    if x.shape[0] != T or wt.shape != (x.shape[1], N):
        raise ValueError("dy must be T x N, x T x K and wt K x N")
    _one_device(dy, x, wt)
    if _elsewhere(dy, stream):
        with _on(dy, stream):
            return mx_linear_backward(dy, x, wt)
    dy_rows, dy_cols = mx_quantize_both(dy)
    dx = mx_mul_mat(dy_rows, wt, dy.dtype)
    return dx, mx_mul_mat(dy_cols, mx_quantize(x, axis=0), torch.float32)


def mx_moe(x, router, gate_up: MXMatrix, down: MXMatrix, top_k: int, renormalize: bool = True, out=None, stream=None):
    """A mixture-of-experts layer for a few tokens (retro_moe): x is T x D,
    router E x D (float32 or x's type), gate_up E * 2F x D (each expert's F
    gate rows, then its F up rows) and down E * D x F, both microscaled. Each
    token goes to the top_k experts of largest x . router[e], whose outputs
    down (silu(gate x) * (up x)) are added with softmax shares: over the
    chosen experts (renormalize) or over all. Returns T x D of x's type."""
    xtype, ldx = _floats(x, "x")
    rtype, ldr = _floats(router, "router")
    _matrix(gate_up, "gate_up")
    _matrix(down, "down")
    T, D = x.shape
    E, F = router.shape[0], down.K
    if router.shape[1] != D or gate_up.rows != E * 2 * F or gate_up.K != D or down.rows != E * D:
        raise ValueError("router must be E x D, gate_up E * 2F x D and down E * D x F")
    _one_device(x, router, gate_up, down)
    if _elsewhere(x, stream):
        with _on(x, stream):
            return mx_moe(x, router, gate_up, down, top_k, renormalize, out)
    if out is None:
        out, ld = torch.empty((T, D), dtype=x.dtype, device=x.device), D
    else:
        ld = _given(out, T, D, x.dtype, x)
    need = _moe_workspace(xtype, T, D, F, E, top_k)
    if need < 0:
        _check(need)
    ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
    _check(lib.retro_moe(xtype, x.data_ptr(), ldx, rtype, router.data_ptr(), ldr, *gate_up._planes(),
                         *down._planes(), out.data_ptr(), ld, T, D, F, E, top_k, int(bool(renormalize)),
                         None if ws is None else ws.data_ptr(), need, _handle()))
    return out
