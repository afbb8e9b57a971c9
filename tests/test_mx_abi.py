"""Refusals of the microscaled 4-bit operators and the expert layer: every one
is made on the host before a device is touched, so these need no GPU and pass
addresses that are never read."""

import pytest
import torch

q = pytest.importorskip("quantized_weight_backward_amd")

A = 1 << 20  # 16-byte aligned addresses, far enough apart not to overlap


def addr(i):
    return A + i * (1 << 40)


def quantize(**k):
    a = dict(type=q.MXFP4, xtype=q.F32, X=addr(1), ldx=64, W=addr(2), K=64, N=8) | k
    return q.lib.retro_quantize(a["type"], a["xtype"], a["X"], a["ldx"], a["W"], a["K"], a["N"], None)


@pytest.mark.parametrize("change,code", [
    (dict(type=q.Q4_0), q.E_TYPE), (dict(type=77), q.E_TYPE), (dict(xtype=q.Q8_0), q.E_TYPE),
    (dict(K=48), q.E_SHAPE), (dict(type=q.NVFP4, K=32), q.E_SHAPE), (dict(K=-32), q.E_SHAPE),
    (dict(N=-1), q.E_SHAPE), (dict(N=1 << 31), q.E_SHAPE), (dict(ldx=63), q.E_SHAPE),
    (dict(ldx=1 << 60), q.E_SHAPE), (dict(X=None), q.E_NULL), (dict(W=None), q.E_NULL),
    (dict(W=addr(2) + 8), q.E_ALIGN), (dict(X=addr(1) + 2), q.E_ALIGN), (dict(W=addr(1) + 64), q.E_ALIAS),
    (dict(N=0, X=None, W=None), q.OK), (dict(K=0, X=None, W=None), q.OK)])
def test_quantize(change, code):
    assert quantize(**change) == code


def mx_quantize(**k):
    a = dict(xtype=q.BF16, X=addr(1), ldx=300, rows=70, cols=300, rc=addr(2), rs=addr(3), cc=addr(4), cs=addr(5)) | k
    return q.lib.retro_mx_quantize(a["xtype"], a["X"], a["ldx"], a["rows"], a["cols"], a["rc"], a["rs"], a["cc"],
                                   a["cs"], None)


@pytest.mark.parametrize("change,code", [
    (dict(xtype=q.MXFP4), q.E_TYPE), (dict(rows=-1), q.E_SHAPE), (dict(cols=1 << 31, ldx=1 << 31), q.E_SHAPE),
    (dict(ldx=299), q.E_SHAPE), (dict(X=None), q.E_NULL), (dict(rc=None), q.E_NULL), (dict(cs=None), q.E_NULL),
    (dict(rc=None, rs=None, cc=None, cs=None), q.E_NULL), (dict(X=addr(1) + 1), q.E_ALIGN),
    (dict(rs=addr(3) + 8), q.E_ALIGN), (dict(cc=addr(4) + 4), q.E_ALIGN), (dict(rc=addr(1) + 1600), q.E_ALIAS),
    (dict(cc=addr(2)), q.E_ALIAS), (dict(cs=addr(3) + 16), q.E_ALIAS),
    (dict(rows=0, X=None, rc=None, rs=None, cc=None, cs=None), q.OK)])
def test_mx_quantize(change, code):
    assert mx_quantize(**change) == code


def dequantize(**k):
    a = dict(ytype=q.F16, codes=addr(1), scales=addr(2), Y=addr(3), ldy=300, K=300, rows=9) | k
    return q.lib.retro_mx_dequantize(a["ytype"], a["codes"], a["scales"], a["Y"], a["ldy"], a["K"], a["rows"], None)


@pytest.mark.parametrize("change,code", [
    (dict(ytype=5), q.E_TYPE), (dict(rows=-1), q.E_SHAPE), (dict(ldy=299), q.E_SHAPE), (dict(codes=None), q.E_NULL),
    (dict(Y=None), q.E_NULL), (dict(codes=addr(1) + 8), q.E_ALIGN), (dict(Y=addr(3) + 1), q.E_ALIGN),
    (dict(Y=addr(2) + 16), q.E_ALIAS), (dict(rows=0, codes=None, scales=None, Y=None), q.OK)])
def test_mx_dequantize(change, code):
    assert dequantize(**change) == code


@pytest.mark.parametrize("args,code", [
    ((addr(1), addr(2), addr(3), 48, 4), q.E_SHAPE), ((addr(1), addr(2), addr(3), 64, -4), q.E_SHAPE),
    ((None, addr(2), addr(3), 64, 4), q.E_NULL), ((addr(1) + 8, addr(2), addr(3), 64, 4), q.E_ALIGN),
    ((addr(1), addr(1) + 16, addr(3), 64, 4), q.E_ALIAS), ((None, None, None, 64, 0), q.OK)])
def test_mx_from_blocks(args, code):
    assert q.lib.retro_mx_from_blocks(*args, None) == code


def product(**k):
    a = dict(ytype=q.F32, ac=addr(1), as_=addr(2), bc=addr(3), bs=addr(4), Y=addr(5), ldy=50, K=300, N=50, T=20) | k
    return q.lib.retro_mx_mul_mat(a["ytype"], a["ac"], a["as_"], a["bc"], a["bs"], a["Y"], a["ldy"], a["K"], a["N"],
                                  a["T"], None)


@pytest.mark.parametrize("change,code", [
    (dict(ytype=q.Q4_K), q.E_TYPE), (dict(K=-1), q.E_SHAPE), (dict(ldy=49), q.E_SHAPE), (dict(T=1 << 31), q.E_SHAPE),
    (dict(T=(1 << 31) - 1, N=(1 << 31) - 1, ldy=(1 << 31) - 1), q.E_SHAPE), (dict(ac=None), q.E_NULL),
    (dict(bs=None), q.E_NULL), (dict(Y=None), q.E_NULL), (dict(as_=addr(2) + 8), q.E_ALIGN),
    (dict(Y=addr(5) + 2), q.E_ALIGN), (dict(Y=addr(1) + 32), q.E_ALIAS), (dict(Y=addr(4)), q.E_ALIAS),
    (dict(T=0, ac=None, as_=None, bc=None, bs=None, Y=None), q.OK)])
def test_mx_mul_mat(change, code):
    assert product(**change) == code


def test_mx_variants():
    args = (q.F32, addr(1), addr(2), addr(3), addr(4), addr(5), 50, 300, 50, 20, None)
    assert q.lib.retro_mx_mul_mat_variant(99, *args) == q.E_VARIANT
    assert q.lib.retro_mx_mul_mat_variant(-1, *args) == q.E_VARIANT
    K = 1 << 30  # 256 rows of codes pass 32 bits: the simple kernel alone
    assert q.MX_VARIANT_NAMES[q.mx_mul_mat_choice(K, 100, 300)] == "simple"
    big = (q.F32, addr(1), addr(2), addr(3), addr(4), addr(5), 50, K, 50, 20, None)
    for variant, name in q.MX_VARIANT_NAMES.items():
        if name.startswith("tile"):
            assert q.lib.retro_mx_mul_mat_variant(variant, *big) == q.E_VARIANT
    assert q.lib.retro_mx_mul_mat_choice(q.Q4_0, 50, 300, 50, 20) == q.E_TYPE
    assert q.lib.retro_mx_mul_mat_choice(q.F32, 49, 300, 50, 20) == q.E_SHAPE


def linear(**k):
    a = dict(xtype=q.BF16, X=addr(1), ldx=3000, bc=addr(3), bs=addr(4), Y=addr(5), ldy=500, K=3000, N=500, T=200,
             ws=addr(6), n=1 << 30) | k
    return q.lib.retro_mx_linear(a["xtype"], a["X"], a["ldx"], a["bc"], a["bs"], a["Y"], a["ldy"], a["K"], a["N"],
                                 a["T"], a["ws"], a["n"], None)


@pytest.mark.parametrize("change,code", [
    (dict(xtype=q.MXFP4), q.E_TYPE), (dict(ldx=2999), q.E_SHAPE), (dict(N=-1), q.E_SHAPE), (dict(X=None), q.E_NULL),
    (dict(bc=None), q.E_NULL), (dict(X=addr(1) + 1), q.E_ALIGN), (dict(bs=addr(4) + 4), q.E_ALIGN),
    (dict(Y=addr(1) + 32), q.E_ALIAS), (dict(ws=None), q.E_WORKSPACE), (dict(n=1000), q.E_WORKSPACE),
    (dict(ws=addr(6) + 8), q.E_WORKSPACE), (dict(ws=addr(5)), q.E_WORKSPACE), (dict(ws=addr(3)), q.E_WORKSPACE),
    (dict(T=0, X=None, bc=None, bs=None, Y=None, ws=None, n=0), q.OK)])
def test_mx_linear(change, code):
    assert linear(**change) == code


def moe(**k):
    a = dict(xtype=q.BF16, X=addr(1), ldx=96, rtype=q.F32, R=addr(2), ldr=96, gc=addr(3), gs=addr(4), dc=addr(5),
             ds=addr(6), Y=addr(7), ldy=96, T=4, D=96, F=40, E=8, k=2, ws=addr(8), n=1 << 30) | k
    return q.lib.retro_moe(a["xtype"], a["X"], a["ldx"], a["rtype"], a["R"], a["ldr"], a["gc"], a["gs"], a["dc"],
                           a["ds"], a["Y"], a["ldy"], a["T"], a["D"], a["F"], a["E"], a["k"], 1, a["ws"], a["n"], None)


@pytest.mark.parametrize("change,code", [
    (dict(xtype=q.Q4_0), q.E_TYPE), (dict(rtype=q.F16), q.E_TYPE), (dict(T=65), q.E_SHAPE), (dict(T=-1), q.E_SHAPE),
    (dict(E=257), q.E_SHAPE), (dict(E=0), q.E_SHAPE), (dict(k=0), q.E_SHAPE), (dict(k=9), q.E_SHAPE),
    (dict(E=64, k=17), q.E_SHAPE), (dict(D=0, ldx=0, ldy=0, ldr=0), q.E_SHAPE), (dict(F=0), q.E_SHAPE),
    (dict(F=1 << 30), q.E_SHAPE), (dict(ldx=95), q.E_SHAPE), (dict(ldr=95), q.E_SHAPE), (dict(ldy=95), q.E_SHAPE),
    (dict(X=None), q.E_NULL), (dict(R=None), q.E_NULL), (dict(ds=None), q.E_NULL), (dict(Y=None), q.E_NULL),
    (dict(R=addr(2) + 2), q.E_ALIGN), (dict(gc=addr(3) + 8), q.E_ALIGN), (dict(Y=addr(1) + 64), q.E_ALIAS),
    (dict(Y=addr(5)), q.E_ALIAS), (dict(ws=None), q.E_WORKSPACE), (dict(n=100), q.E_WORKSPACE),
    (dict(ws=addr(7)), q.E_WORKSPACE), (dict(ws=addr(8) + 4), q.E_WORKSPACE),
    (dict(T=0, X=None, R=None, Y=None, ws=None, n=0), q.OK)])
def test_moe(change, code):
    assert moe(**change) == code


def test_sizes():
    assert q.lib.retro_mx_code_bytes(3, 257) == 3 * 256 and q.lib.retro_mx_scale_bytes(3, 257) == 3 * 16
    assert q.lib.retro_mx_code_bytes(-1, 5) == -1 and q.lib.retro_mx_scale_bytes(5, 1 << 31) == -1
    assert q.lib.retro_mx_linear_workspace_size(q.Q4_0, 1, 1, 1) == q.E_TYPE
    assert q.lib.retro_mx_linear_workspace_size(q.F32, -1, 1, 1) == q.E_SHAPE
    assert q.lib.retro_moe_workspace_size(q.F32, 65, 1, 1, 1, 1) == q.E_SHAPE
    assert q.lib.retro_moe_workspace_size(q.F32, 0, 1, 1, 1, 1) == 0
    assert q.lib.retro_moe_workspace_size(q.BF16, 8, 96, 40, 8, 2) % 16 == 0


def test_the_binding_refuses_host_tensors_and_wrong_arguments():
    x = torch.zeros((4, 64))
    for call in (lambda: q.quantize(q.MXFP4, x), lambda: q.mx_quantize(x), lambda: q.mx_quantize(x, axis=2),
                 lambda: q.MXMatrix(x, x, 64), lambda: q.mx_linear(x, x), lambda: q.mx_mul_mat(x, x),
                 lambda: q.mx_dequantize(x), lambda: q.mx_from_blocks(x, 64, 4),
                 lambda: q.mx_linear_backward(x, x, x), lambda: q.mx_moe(x, x, x, x, 1)):
        with pytest.raises(ValueError):
            call()


def test_sizes_past_one_launch():
    """A launch takes fewer than 2^32 threads: tiles that need more are refused
    or passed over, and all calls agree on the sizes they take."""
    T, N = 1 << 19, 1 << 20  # 2^23 workgroups of 512 threads and 256 x 256 outputs
    args = (q.F32, addr(1), addr(2), addr(3), addr(4), addr(5), N, 256, N, T, None)
    for variant, name in q.MX_VARIANT_NAMES.items():
        if name.startswith("tile"):
            assert q.lib.retro_mx_mul_mat_variant(variant, *args) == q.E_VARIANT, name
    assert q.MX_VARIANT_NAMES[q.mx_mul_mat_choice(256, N, T)] == "simple"
    assert q.MX_VARIANT_NAMES[q.mx_mul_mat_choice(256, (1 << 31) - 1, 32)] == "skinny"
    assert q.MX_VARIANT_NAMES[q.mx_mul_mat_choice(256, N // 2, T)].startswith("tile")
    most = (1 << 31) - 1
    assert product(T=most, N=most, ldy=most) == q.E_SHAPE
    assert linear(T=most, N=most, ldy=most) == q.E_SHAPE
    assert q.lib.retro_mx_mul_mat_choice(q.F32, most, 300, most, most) == q.E_SHAPE
    assert q.lib.retro_mx_linear_workspace_size(q.F32, 300, most, most) == q.E_SHAPE


@pytest.mark.parametrize("dtype,T,N,K,name", [
    (torch.bfloat16, 4096, 14336, 4096, "tile_256x256"), (torch.float32, 8192, 8192, 8192, "tile_256x256"),
    (torch.bfloat16, 2048, 5120, 17408, "tile_256x192"), (torch.float32, 17408, 5120, 2048, "tile_128x128"),
    (torch.bfloat16, 512, 14336, 4096, "tile_128x128"), (torch.bfloat16, 1024, 4096, 4096, "tile_64x128"),
    (torch.bfloat16, 512, 4096, 4096, "tile_64x64"), (torch.bfloat16, 256, 4096, 14336, "tile_64x64_k4"),
    (torch.float16, 333, 1000, 1500, "tile_32x64_k4"), (torch.bfloat16, 32, 14336, 4096, "tile_32x64_k4"),
    (torch.bfloat16, 16, 4096, 14336, "skinny"), (torch.bfloat16, 64, 4096, 1 << 30, "simple")])
def test_kernels_chosen(dtype, T, N, K, name):
    assert q.MX_VARIANT_NAMES[q.mx_mul_mat_choice(K, N, T, dtype)] == name


def test_the_largest_layers():
    most = (1 << 22) - 1
    assert q.lib.retro_moe_workspace_size(q.BF16, 1, most, most, 4, 2) > 0
    assert q.lib.retro_moe_workspace_size(q.BF16, 1, most + 1, 40, 4, 2) == q.E_SHAPE
    assert q.lib.retro_moe_workspace_size(q.BF16, 1, 40, most + 1, 4, 2) == q.E_SHAPE
