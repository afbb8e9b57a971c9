"""Refusals of the operators over a vocabulary: every one is made on the host before
a device is touched, so these need no GPU and pass addresses that are never read."""

import pytest

q = pytest.importorskip("quantized_weight_backward_amd")

A = 1 << 20  # 16-byte aligned addresses, far enough apart not to overlap
I32, I64 = 26, 27
NONE = dict(W=None, X=None, Y=None, ids=None, ws=None)


def addr(i):
    return A + i * (1 << 40)


def embedding(**k):
    a = dict(type=q.Q8_0, W=addr(1), ldw=68, idtype=I64, ids=addr(2), ytype=q.BF16, Y=addr(3), ldy=64, K=64, N=100, T=9) | k
    return q.lib.retro_embedding(a["type"], a["W"], a["ldw"], a["idtype"], a["ids"], 1.0, a["ytype"], a["Y"], a["ldy"],
                                 a["K"], a["N"], a["T"], None)


@pytest.mark.parametrize("change,code", [
    (dict(type=77), q.E_TYPE), (dict(ytype=q.Q8_0), q.E_TYPE), (dict(idtype=25), q.E_TYPE), (dict(K=48), q.E_SHAPE),
    (dict(K=-32), q.E_SHAPE), (dict(K=1 << 22, ldw=1 << 23, ldy=1 << 22), q.E_SHAPE), (dict(N=-1), q.E_SHAPE),
    (dict(N=1 << 31), q.E_SHAPE), (dict(T=-1), q.E_SHAPE), (dict(T=1 << 31), q.E_SHAPE), (dict(ldw=66), q.E_SHAPE),
    (dict(ldw=1 << 60), q.E_SHAPE), (dict(ldy=63), q.E_SHAPE), (dict(ldy=1 << 62), q.E_SHAPE), (dict(W=None), q.E_NULL),
    (dict(ids=None), q.E_NULL), (dict(Y=None), q.E_NULL), (dict(W=addr(1) + 8), q.E_ALIGN),
    (dict(Y=addr(3) + 1), q.E_ALIGN), (dict(ids=addr(2) + 4), q.E_ALIGN), (dict(ldw=69), q.E_ALIGN),
    (dict(Y=addr(1) + 6798), q.E_ALIAS), (dict(Y=addr(2) + 70), q.E_ALIAS),
    (dict(T=0, W=None, Y=None, ids=None), q.OK), (dict(K=0, W=None, Y=None, ids=None), q.OK)])
def test_embedding(change, code):
    assert embedding(**change) == code


def embedding_backward(**k):
    a = dict(idtype=I32, ids=addr(1), ytype=q.F16, Y=addr(2), ldy=70, wtype=q.F32, W=addr(3), ldw=64, add=0, K=64, N=50, T=300,
             ws=addr(4), nbytes=None) | k
    need = q.lib.retro_embedding_backward_workspace_size(a["K"], a["N"], a["T"])
    return q.lib.retro_embedding_backward(a["idtype"], a["ids"], a["ytype"], a["Y"], a["ldy"], 1.0, a["wtype"], a["W"],
                                          a["ldw"], a["add"], a["K"], a["N"], a["T"], a["ws"],
                                          need if a["nbytes"] is None else need + a["nbytes"], None)


@pytest.mark.parametrize("change,code", [
    (dict(ytype=q.Q4_0), q.E_TYPE), (dict(wtype=q.Q4_0), q.E_TYPE), (dict(idtype=0), q.E_TYPE), (dict(K=-1), q.E_SHAPE),
    (dict(K=1 << 22, ldy=1 << 22, ldw=1 << 22), q.E_SHAPE), (dict(N=1 << 31), q.E_SHAPE), (dict(T=1 << 28), q.E_SHAPE),
    (dict(ldy=63), q.E_SHAPE), (dict(ldw=63), q.E_SHAPE), (dict(ldw=1 << 61), q.E_SHAPE), (dict(ids=None), q.E_NULL),
    (dict(Y=None), q.E_NULL), (dict(W=None), q.E_NULL), (dict(W=addr(3) + 2), q.E_ALIGN), (dict(Y=addr(2) + 1), q.E_ALIGN),
    (dict(ids=addr(1) + 2), q.E_ALIGN), (dict(W=addr(2) + 64), q.E_ALIAS), (dict(W=addr(1)), q.E_ALIAS),
    (dict(ws=None), q.E_WORKSPACE), (dict(ws=addr(4) + 8), q.E_WORKSPACE), (dict(nbytes=-1), q.E_WORKSPACE),
    (dict(ws=addr(3) + 12784), q.E_WORKSPACE), (dict(ws=addr(2)), q.E_WORKSPACE), (dict(ws=addr(1)), q.E_WORKSPACE),
    (dict(N=0, ids=None, Y=None, W=None, ws=None), q.OK), (dict(K=0, ids=None, Y=None, W=None, ws=None), q.OK),
    (dict(T=0, add=1, ids=None, Y=None, W=None, ws=None), q.OK)])
def test_embedding_backward(change, code):
    assert embedding_backward(**change) == code


def cross_entropy(**k):
    a = dict(type=q.BF16, W=addr(1), ldw=128, xtype=q.BF16, X=addr(2), ldx=64, idtype=I64, t=addr(3), loss=addr(4),
             lse=addr(5), K=64, N=1000, T=70, ws=addr(6), nbytes=0) | k
    need = q.lib.retro_cross_entropy_workspace_size(a["type"], a["ldw"], a["xtype"], a["K"], a["N"], a["T"])
    return q.lib.retro_cross_entropy(a["type"], a["W"], a["ldw"], a["xtype"], a["X"], a["ldx"], a["idtype"], a["t"],
                                     a["loss"], a["lse"], a["K"], a["N"], a["T"], a["ws"], need + a["nbytes"], None)


COMMON = [
    (dict(type=77), q.E_TYPE), (dict(xtype=q.Q4_0), q.E_TYPE), (dict(idtype=3), q.E_TYPE), (dict(K=-1), q.E_SHAPE),
    (dict(type=q.Q8_0, K=48), q.E_SHAPE), (dict(K=1 << 22, ldw=1 << 24, ldx=1 << 22), q.E_SHAPE), (dict(N=-1), q.E_SHAPE),
    (dict(N=1 << 31), q.E_SHAPE), (dict(T=1 << 22), q.E_SHAPE), (dict(ldw=126), q.E_SHAPE), (dict(ldw=1 << 61), q.E_SHAPE),
    (dict(ldx=63), q.E_SHAPE), (dict(W=None), q.E_NULL), (dict(X=None), q.E_NULL), (dict(t=None), q.E_NULL),
    (dict(lse=None), q.E_NULL), (dict(W=addr(1) + 8), q.E_ALIGN), (dict(X=addr(2) + 1), q.E_ALIGN),
    (dict(t=addr(3) + 4), q.E_ALIGN), (dict(lse=addr(5) + 2), q.E_ALIGN), (dict(ldw=129), q.E_ALIGN),
    (dict(ws=None), q.E_WORKSPACE), (dict(ws=addr(6) + 4), q.E_WORKSPACE), (dict(nbytes=-1), q.E_WORKSPACE),
    (dict(ws=addr(1)), q.E_WORKSPACE), (dict(ws=addr(2) + 64), q.E_WORKSPACE), (dict(ws=addr(3)), q.E_WORKSPACE),
    (dict(ws=addr(5)), q.E_WORKSPACE)]


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(loss=None), q.E_NULL), (dict(loss=addr(4) + 1), q.E_ALIGN), (dict(loss=addr(5)), q.E_ALIAS),
    (dict(loss=addr(2)), q.E_ALIAS), (dict(lse=addr(1) + 64), q.E_ALIAS), (dict(lse=addr(3)), q.E_ALIAS),
    (dict(ws=addr(4)), q.E_WORKSPACE),
    (dict(T=0, W=None, X=None, t=None, loss=None, lse=None, ws=None), q.OK)])
def test_cross_entropy(change, code):
    assert cross_entropy(**change) == code


def cross_entropy_backward(**k):
    a = dict(type=q.BF16, W=addr(1), ldw=128, xtype=q.BF16, X=addr(2), ldx=64, idtype=I64, t=addr(3), lse=addr(5),
             g=addr(7), dX=addr(8), lddx=64, dW=addr(9), lddw=64, K=64, N=1000, T=70, ws=addr(6), nbytes=0) | k
    need = q.lib.retro_cross_entropy_backward_workspace_size(a["type"], a["ldw"], a["xtype"], int(bool(a["dW"])), a["K"],
                                                             a["N"], a["T"])
    return q.lib.retro_cross_entropy_backward(a["type"], a["W"], a["ldw"], a["xtype"], a["X"], a["ldx"], a["idtype"],
                                              a["t"], a["lse"], a["g"], a["dX"], a["lddx"], a["dW"], a["lddw"], a["K"],
                                              a["N"], a["T"], a["ws"], need + a["nbytes"], None)


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(type=q.Q8_0, ldw=68), q.E_TYPE), (dict(lddx=63), q.E_SHAPE), (dict(lddw=63), q.E_SHAPE), (dict(g=None), q.E_NULL),
    (dict(dX=None, dW=None), q.E_NULL), (dict(g=addr(7) + 2), q.E_ALIGN), (dict(dX=addr(8) + 1), q.E_ALIGN),
    (dict(dW=addr(9) + 1), q.E_ALIGN), (dict(dX=addr(2)), q.E_ALIAS), (dict(dW=addr(1)), q.E_ALIAS),
    (dict(dX=addr(9)), q.E_ALIAS), (dict(dX=addr(7)), q.E_ALIAS), (dict(dW=addr(5)), q.E_ALIAS),
    (dict(ws=addr(8)), q.E_WORKSPACE), (dict(ws=addr(9)), q.E_WORKSPACE), (dict(ws=addr(7)), q.E_WORKSPACE),
    (dict(K=0, X=None, W=None, dX=None, dW=None, ws=None), q.OK),
    (dict(T=0, dW=None, X=None, t=None, lse=None, g=None, dX=None, ws=None), q.OK),
    (dict(T=0, N=0, X=None, t=None, lse=None, g=None, dX=None, ws=None), q.OK)])
def test_cross_entropy_backward(change, code):
    assert cross_entropy_backward(**change) == code


def test_workspace_sizes():
    """No size depends on the tokens beyond growing with them, and none holds the logits."""
    f, b = q.lib.retro_cross_entropy_workspace_size, q.lib.retro_cross_entropy_backward_workspace_size
    e = q.lib.retro_embedding_backward_workspace_size
    for type, ldw in ((q.BF16, 8192), (q.Q4_K, 2304), (q.F32, 16384)):
        for T in (1, 64, 65, 4096):
            assert 0 < f(type, ldw, q.BF16, 4096, 1 << 20, T) < 4 * T * (1 << 20) + (1 << 30)
            assert b(type, ldw, q.BF16, 0, 4096, 1 << 20, T) > 0
    assert f(q.BF16, 8192, q.BF16, 4096, 131072, 4096) < 1 << 27
    assert f(q.BF16, 128, q.BF16, 64, 100, 0) == 0 and b(q.BF16, 128, q.BF16, 1, 64, 0, 5) == 0
    assert b(q.Q8_0, 68, q.BF16, 1, 64, 10, 5) == q.E_TYPE and f(q.BF16, 2, q.BF16, 64, 10, 5) == q.E_SHAPE
    assert e(64, 10, 0) == 0 and e(64, 10, 1) > 0 and e(0, 10, 5) == 0 and e(64, 0, 5) == 0 and e(-1, 1, 1) == q.E_SHAPE
    assert e(4096, 131072, 16384) < 1 << 24
