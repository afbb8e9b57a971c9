"""Binding of the operators over a model's vocabulary (include/retro_vocab.h):
marshals torch tensors into the C ABI and nothing else.

    embedding               rows of a resident table, of floats or packed blocks
    embedding_backward      its gradient with respect to a float table
    cross_entropy           softmax cross entropy through a resident head, no logits kept
    cross_entropy_backward  its gradients with respect to the tokens and a float head

A table W of N rows x K is a 2-D uint8 tensor or view of N rows whose first
row_bytes(wtype, K) bytes hold a row; or, without such rows, a contiguous device tensor
of N * row_bytes bytes; one of floats also a 2-D view of its own dtype with contiguous
rows. Ids and targets are 1-D contiguous int32 or int64 device tensors;
a value outside 0 .. N - 1 is no token (padding, or not learnt from).

Every call runs asynchronously on `stream` (default: torch's current stream of the
operands' device); outputs and scratch it allocates belong to that stream. None is
recorded for autograd: results require no gradient, and a training step calls the
_backward functions.
"""

from __future__ import annotations

import functools

import torch

from . import BF16, E_SHAPE, E_TYPE, F16, F32, TYPES, _check, _device_tensor, _row_stride, lib, row_bytes
from .mx import _FLOAT, _elsewhere, _floats, _given, _handle, _on, _one_device

_IDS = {torch.int32: 26, torch.int64: 27}
_DTYPES = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}


def _table(wtype, W, K):
    """(rows, bytes between rows) of a table."""
    _device_tensor(W, "W", contiguous=False)
    rb = row_bytes(wtype, K)
    if rb < 0:
        _check(E_SHAPE if wtype in TYPES.values() else E_TYPE)
    if rb == 0:
        raise ValueError("K must be positive")
    if W.dim() == 2 and W.dtype == _DTYPES.get(wtype) and W.shape[1] == K:
        return W.shape[0], _row_stride(W, "W") * W.element_size()
    if W.dim() == 2 and W.dtype == torch.uint8 and W.shape[1] >= rb:
        ldw = _row_stride(W, "W")
        return W.shape[0], (ldw if W.shape[0] > 1 else rb)
    if W.is_contiguous():
        nbytes = W.numel() * W.element_size()
        if nbytes % rb:
            raise ValueError(f"W holds {nbytes} bytes, no whole number of rows of {rb}")
        return nbytes // rb, rb
    raise ValueError(f"a strided W must be a uint8 view of rows of at least {rb} bytes")


def _tokens(t, name, T=None):
    _device_tensor(t, name)
    code = _IDS.get(t.dtype)
    if code is None or t.dim() != 1:
        raise ValueError(f"{name} must be a 1-D int32 or int64 tensor")
    if T is not None and t.shape[0] != T:
        raise ValueError(f"{name} must hold {T} values")
    return code


def _vector(t, name, T):
    _device_tensor(t, name)
    if t.dtype != torch.float32 or t.shape != (T,):
        raise ValueError(f"{name} must be float32 of shape {(T,)}")


# sizes of shapes that come again and again
@functools.lru_cache(maxsize=1024)
def _embedding_backward_workspace(K: int, N: int, T: int) -> int:
    return lib.retro_embedding_backward_workspace_size(K, N, T)


@functools.lru_cache(maxsize=1024)
def _forward_workspace(wtype: int, ldw: int, xtype: int, K: int, N: int, T: int) -> int:
    return lib.retro_cross_entropy_workspace_size(wtype, ldw, xtype, K, N, T)


@functools.lru_cache(maxsize=1024)
def _backward_workspace(wtype: int, ldw: int, xtype: int, weight_grad: bool, K: int, N: int, T: int) -> int:
    return lib.retro_cross_entropy_backward_workspace_size(wtype, ldw, xtype, weight_grad, K, N, T)


def _scratch(need, device):
    _check(min(need, 0))
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


def _at(t):
    return None if t is None else t.data_ptr()


def embedding(wtype: int, W, ids, K: int, scale: float = 1.0, dtype=torch.float32, out=None, stream=None):
    """Y[t] = scale * W[ids[t]] (T x K of dtype), a row of zeros where ids[t] is no token."""
    N, ldw = _table(wtype, W, K)
    idtype = _tokens(ids, "ids")
    ytype = _FLOAT.get(dtype)
    if ytype is None:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    _one_device(W, ids)
    if _elsewhere(W, stream):
        with _on(W, stream):
            return embedding(wtype, W, ids, K, scale, dtype, out)
    T, ld = ids.shape[0], K
    if out is None:
        out = torch.empty((T, K), dtype=dtype, device=W.device)
    else:
        ld = _given(out, T, K, dtype, W)
    _check(lib.retro_embedding(wtype, W.data_ptr(), ldw, idtype, ids.data_ptr(), scale, ytype, out.data_ptr(), ld, K, N,
                               T, _handle()))
    return out


def embedding_backward(ids, dy, N: int, scale: float = 1.0, dtype=torch.float32, out=None, accumulate: bool = False,
                       stream=None):
    """The gradient of embedding with respect to a float table of N rows, from the
    gradient dy (T x K) of its result: dW[n] = scale * the sum of dy[t] over the t
    with ids[t] = n (N x K of dtype). With accumulate it is added to `out`, of which
    then only the rows that a token has are touched."""
    idtype = _tokens(ids, "ids")
    ytype, ldy = _floats(dy, "dy")
    T, K = dy.shape
    if ids.shape[0] != T:
        raise ValueError("ids and the rows of dy must be as many")
    if out is not None:
        dtype = out.dtype if accumulate else dtype
    elif accumulate:
        raise ValueError("accumulate needs out")
    wtype = _FLOAT.get(dtype)
    if wtype is None:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    _one_device(dy, ids)
    if _elsewhere(dy, stream):
        with _on(dy, stream):
            return embedding_backward(ids, dy, N, scale, dtype, out, accumulate)
    ld = K
    if out is None:
        out = torch.empty((N, K), dtype=dtype, device=dy.device)
    else:
        ld = _given(out, N, K, dtype, dy)
    need = _embedding_backward_workspace(K, N, T)
    ws = _scratch(need, dy.device)
    _check(lib.retro_embedding_backward(idtype, ids.data_ptr(), ytype, dy.data_ptr(), ldy, scale, wtype, out.data_ptr(),
                                        ld, int(bool(accumulate)), K, N, T, _at(ws), need, _handle()))
    return out


def cross_entropy(wtype: int, W, x, targets, stream=None):
    """(loss, lse), float32 of T values each: with the logits l = x W^T of T x K
    tokens x, lse[t] = log sum_n exp l[t][n] and loss[t] = lse[t] - l[t][targets[t]],
    0 where targets[t] is no token. The logits are never held."""
    xtype, ldx = _floats(x, "x")
    T, K = x.shape
    N, ldw = _table(wtype, W, K)
    idtype = _tokens(targets, "targets", T)
    _one_device(x, W, targets)
    if _elsewhere(x, stream):
        with _on(x, stream):
            return cross_entropy(wtype, W, x, targets)
    both = torch.empty((2, T), dtype=torch.float32, device=x.device)
    loss, lse = both[0], both[1]
    need = _forward_workspace(wtype, ldw, xtype, K, N, T)
    ws = _scratch(need, x.device)
    _check(lib.retro_cross_entropy(wtype, W.data_ptr(), ldw, xtype, x.data_ptr(), ldx, idtype, targets.data_ptr(),
                                   loss.data_ptr(), lse.data_ptr(), K, N, T, _at(ws), need, _handle()))
    return loss, lse


def cross_entropy_backward(wtype: int, W, x, targets, lse, dloss, weight_grad: bool = False, dx_out=None, dw_out=None,
                           stream=None):
    """(dx, dw) from lse as cross_entropy gave it and the gradient dloss (float32 of
    T values) of its loss: dx T x K of x's dtype, and, with weight_grad, dw N x K of
    the float table's (None otherwise). Tokens whose target is none have dx = 0 and no
    part in dw. A packed table is frozen: it has no gradient."""
    xtype, ldx = _floats(x, "x")
    T, K = x.shape
    N, ldw = _table(wtype, W, K)
    idtype = _tokens(targets, "targets", T)
    _vector(lse, "lse", T)
    _vector(dloss, "dloss", T)
    if weight_grad and wtype not in _DTYPES:
        _check(E_TYPE)
    if dw_out is not None and not weight_grad:
        raise ValueError("dw_out needs weight_grad")
    _one_device(x, W, targets, lse, dloss)
    if _elsewhere(x, stream):
        with _on(x, stream):
            return cross_entropy_backward(wtype, W, x, targets, lse, dloss, weight_grad, dx_out, dw_out)
    lddx = lddw = K
    if dx_out is None:
        dx_out = torch.empty((T, K), dtype=x.dtype, device=x.device)
    else:
        lddx = _given(dx_out, T, K, x.dtype, x)
    if weight_grad:
        if dw_out is None:
            dw_out = torch.empty((N, K), dtype=_DTYPES[wtype], device=x.device)
        else:
            lddw = _given(dw_out, N, K, _DTYPES[wtype], x)
    need = _backward_workspace(wtype, ldw, xtype, bool(weight_grad), K, N, T)
    ws = _scratch(need, x.device)
    _check(lib.retro_cross_entropy_backward(wtype, W.data_ptr(), ldw, xtype, x.data_ptr(), ldx, idtype,
                                            targets.data_ptr(), lse.data_ptr(), dloss.data_ptr(), dx_out.data_ptr(),
                                            lddx, _at(dw_out), lddw, K, N, T, _at(ws), need, _handle()))
    return dx_out, dw_out
