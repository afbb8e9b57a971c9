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
"""

from __future__ import annotations

import contextlib

import torch

from . import (BF16, E_SHAPE, E_TYPE, F16, F32, MXFP4, TYPES, _check, _device_tensor, _ptr, _stream_handle, lib,
               row_bytes)

_FLOAT = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
MX_VARIANT_AUTO, MX_VARIANT_SIMPLE, MX_VARIANT_TILE_256x256, MX_VARIANT_TILE_128x128, MX_VARIANT_TILE_64x128, \
    MX_VARIANT_TILE_64x64, MX_VARIANT_SKINNY, MX_VARIANT_TILE_64x64_K4, MX_VARIANT_TILE_32x64_K4 = range(9)
MX_VARIANT_NAMES = {MX_VARIANT_SIMPLE: "simple", MX_VARIANT_TILE_256x256: "tile_256x256",
                    MX_VARIANT_TILE_128x128: "tile_128x128", MX_VARIANT_TILE_64x128: "tile_64x128",
                    MX_VARIANT_TILE_64x64: "tile_64x64", MX_VARIANT_SKINNY: "skinny",
                    MX_VARIANT_TILE_64x64_K4: "tile_64x64_k4", MX_VARIANT_TILE_32x64_K4: "tile_32x64_k4"}
_QUIET = contextlib.nullcontext()


def _on(t, stream):
    """The context of a call on t's device and `stream`: what is allocated in
    it belongs to that stream."""
    if stream is not None:
        return torch.cuda.stream(stream)
    if t.device.index != torch.cuda.current_device():
        return torch.cuda.device(t.device)
    return _QUIET


def _float_type(t, name) -> int:
    code = _FLOAT.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16")
    return code


def _floats(t, name):
    """(type, row stride) of a 2-D float view with contiguous rows."""
    _device_tensor(t, name, contiguous=False)
    code = _float_type(t, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return code, (t.stride(0) if rows > 1 else cols)


def _same_device(*tensors):
    if any(t.device != tensors[0].device for t in tensors[1:]):
        raise ValueError("all operands must be on one device")


def _out(out, shape, dtype, like, name="out"):
    """The output and its row stride."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=like.device), shape[1]
    _device_tensor(out, name, contiguous=False)
    if out.dtype != dtype or tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}")
    _same_device(out, like)
    return out, _floats(out, name)[1]


class MXMatrix:
    """A microscaled 4-bit matrix of `rows` x K: 32 elements along K share a
    power-of-two scale.

    codes   uint8 [rows, ceil(K / 256) * 128]
    scales  uint8 [ceil(K / 256), rows, 8]

    in the layout of include/retro_mx.h (codes past K are zero).
    """

    __slots__ = ("codes", "scales", "K", "rows")

    def __init__(self, codes, scales, K: int):
        _device_tensor(codes, "codes")
        _device_tensor(scales, "scales")
        steps = -(-int(K) // 256)
        if codes.dtype != torch.uint8 or codes.dim() != 2 or codes.shape[1] != steps * 128:
            raise ValueError(f"codes must be uint8 [rows, {steps * 128}] for K = {K}")
        if scales.dtype != torch.uint8 or tuple(scales.shape) != (steps, codes.shape[0], 8):
            raise ValueError(f"scales must be uint8 [{steps}, {codes.shape[0]}, 8]")
        _same_device(codes, scales)
        self.codes, self.scales, self.K, self.rows = codes, scales, int(K), int(codes.shape[0])

    @property
    def shape(self):
        return self.rows, self.K

    @property
    def device(self):
        return self.codes.device

    @staticmethod
    def empty(rows: int, K: int, device):
        steps = -(-K // 256)
        return MXMatrix(torch.empty((rows, steps * 128), dtype=torch.uint8, device=device),
                        torch.empty((steps, rows, 8), dtype=torch.uint8, device=device), K)


def _matrix(m, name):
    if not isinstance(m, MXMatrix):
        raise ValueError(f"{name} must be an MXMatrix")
    return m


def quantize(wtype: int, x, out=None, stream=None):
    """Packed blocks (uint8 [N, row_bytes(wtype, K)]) of an N x K float tensor
    with contiguous rows, wtype MXFP4 or NVFP4."""
    xtype, ldx = _floats(x, "x")
    N, K = x.shape
    rb = row_bytes(wtype, K)
    if rb < 0:
        _check(E_SHAPE if wtype in TYPES.values() else E_TYPE)
    with _on(x, stream):
        if out is None:
            out = torch.empty((N, rb), dtype=torch.uint8, device=x.device)
        else:
            _device_tensor(out, "out")
            if out.dtype != torch.uint8 or out.numel() != N * rb:
                raise ValueError(f"out must hold {N * rb} bytes")
            _same_device(out, x)
        _check(lib.retro_quantize(int(wtype), xtype, _ptr(x), ldx, _ptr(out), K, N, _stream_handle(stream)))
    return out


def _quantize(x, rows: bool, cols: bool, stream):
    xtype, ldx = _floats(x, "x")
    T, K = x.shape
    with _on(x, stream):
        r = MXMatrix.empty(T, K, x.device) if rows else None
        c = MXMatrix.empty(K, T, x.device) if cols else None
        _check(lib.retro_mx_quantize(xtype, _ptr(x), ldx, T, K, _ptr(r.codes) if rows else None,
                                     _ptr(r.scales) if rows else None, _ptr(c.codes) if cols else None,
                                     _ptr(c.scales) if cols else None, _stream_handle(stream)))
    return r, c


def mx_quantize(x, axis: int = 1, stream=None) -> MXMatrix:
    """The microscaled matrix of a 2-D float tensor with contiguous rows:
    axis 1 (or -1) along its rows, axis 0 of its transpose, blocks along the
    columns."""
    if axis not in (0, 1, -1):
        raise ValueError("axis must be 0, 1 or -1")
    r, c = _quantize(x, axis != 0, axis == 0, stream)
    return c if axis == 0 else r


def mx_quantize_both(x, stream=None) -> tuple[MXMatrix, MXMatrix]:
    """mx_quantize along axis 1 and axis 0 from one reading of x."""
    return _quantize(x, True, True, stream)


def mx_dequantize(m: MXMatrix, dtype=torch.float32, out=None, stream=None):
    """The values of a microscaled matrix, rows x K of dtype."""
    _matrix(m, "m")
    if dtype not in _FLOAT:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    with _on(m, stream):
        out, ld = _out(out, m.shape, dtype, m.codes)
        _check(lib.retro_mx_dequantize(_FLOAT[dtype], _ptr(m.codes), _ptr(m.scales), _ptr(out), ld, m.K, m.rows,
                                       _stream_handle(stream)))
    return out


def mx_from_blocks(W, K: int, N: int, stream=None) -> MXMatrix:
    """The microscaled matrix of N rows of packed MXFP4 blocks (same values)."""
    _device_tensor(W, "W")
    rb = row_bytes(MXFP4, K)
    if rb < 0:
        _check(E_SHAPE)
    if W.numel() * W.element_size() != N * rb:
        raise ValueError(f"W holds {W.numel() * W.element_size()} bytes, expected N*row_bytes = {N * rb}")
    with _on(W, stream):
        m = MXMatrix.empty(N, K, W.device)
        _check(lib.retro_mx_from_blocks(_ptr(W), _ptr(m.codes), _ptr(m.scales), int(K), int(N),
                                        _stream_handle(stream)))
    return m


def mx_mul_mat_choice(K: int, N: int, T: int, dtype=torch.float32) -> int:
    """The kernel mx_mul_mat runs for a contiguous T x N result (a key of MX_VARIANT_NAMES)."""
    return int(lib.retro_mx_mul_mat_choice(_FLOAT[dtype], int(N), int(K), int(N), int(T)))


def mx_mul_mat(a: MXMatrix, b: MXMatrix, dtype=torch.float32, out=None, variant: int = MX_VARIANT_AUTO, stream=None):
    """Y[t][n] = sum_k a[t][k] b[n][k] (T x N of dtype)."""
    _matrix(a, "a")
    _matrix(b, "b")
    if a.K != b.K:
        raise ValueError(f"a has K = {a.K}, b has K = {b.K}")
    if dtype not in _FLOAT:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    _same_device(a.codes, b.codes)
    with _on(a, stream):
        out, ld = _out(out, (a.rows, b.rows), dtype, a.codes)
        _check(lib.retro_mx_mul_mat_variant(int(variant), _FLOAT[dtype], _ptr(a.codes), _ptr(a.scales),
                                            _ptr(b.codes), _ptr(b.scales), _ptr(out), ld, a.K, b.rows, a.rows,
                                            _stream_handle(stream)))
    return out


def mx_linear(x, w: MXMatrix, out=None, stream=None):
    """y = x w^T for x a T x K float tensor, quantised along its rows in the
    call; y has x's type."""
    xtype, ldx = _floats(x, "x")
    _matrix(w, "w")
    T, K = x.shape
    if K != w.K:
        raise ValueError(f"x has K = {K}, w has K = {w.K}")
    _same_device(x, w.codes)
    with _on(x, stream):
        out, ld = _out(out, (T, w.rows), x.dtype, x)
        need = lib.retro_mx_linear_workspace_size(xtype, K, w.rows, T)
        ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need > 0 else None
        _check(lib.retro_mx_linear(xtype, _ptr(x), ldx, _ptr(w.codes), _ptr(w.scales), _ptr(out), ld, K, w.rows, T,
                                   _ptr(ws), max(need, 0), _stream_handle(stream)))
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
    _same_device(dy, x, wt.codes)
    with _on(dy, stream):
        dy_rows, dy_cols = mx_quantize_both(dy, stream=stream)
        dx = mx_mul_mat(dy_rows, wt, dy.dtype, stream=stream)
        dw = mx_mul_mat(dy_cols, mx_quantize(x, axis=0, stream=stream), torch.float32, stream=stream)
    return dx, dw


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
    if router.shape[1] != D or gate_up.shape != (E * 2 * F, D) or down.rows != E * D:
        raise ValueError("router must be E x D, gate_up E * 2F x D and down E * D x F")
    _same_device(x, router, gate_up.codes, down.codes)
    with _on(x, stream):
        out, ld = _out(out, (T, D), x.dtype, x)
        need = lib.retro_moe_workspace_size(xtype, T, D, F, E, int(top_k))
        if need < 0:
            _check(need)
        ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
        _check(lib.retro_moe(xtype, _ptr(x), ldx, rtype, _ptr(router), ldr, _ptr(gate_up.codes), _ptr(gate_up.scales),
                             _ptr(down.codes), _ptr(down.scales), _ptr(out), ld, T, D, F, E, int(top_k),
                             int(bool(renormalize)), _ptr(ws), need, _stream_handle(stream)))
    return out
