"""The entry points of the 8-bit product and of the row operators on the CPU: they refuse bad arguments before anything
is launched, size their workspaces, and every kernel that the built-in choice of the product takes is compiled.  No GPU
is used."""
import os

import pytest
import torch

import implicit_gemm_conv_amd as igc

pytestmark = pytest.mark.skipif(not os.path.exists(igc.LIB_PATH), reason="libigc.so not built")

P = 1 << 20  # a 16-byte aligned address that is never dereferenced (validation fails first)
OK, INVALID, MISALIGNED, UNSUPPORTED = igc.IGC_OK, igc.IGC_ERR_INVALID_VALUE, igc.IGC_ERR_MISALIGNED, igc.IGC_ERR_UNSUPPORTED
FAR = 1 << 33

PRODUCT = dict(M=64, N=64, K=64, A=P, lda=64, scale_a=P, B=P, ldb=64, scale_b=P, D=P, ldd=64, d_type=0)


def epi(**kw):
    c = igc.CEpilogue()
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("call,e,expect", [
    (dict(M=-1), None, INVALID), (dict(N=-1), None, INVALID), (dict(K=-1), None, INVALID), (dict(d_type=3), None, INVALID),
    (dict(A=None), None, INVALID), (dict(B=None), None, INVALID), (dict(D=None), None, INVALID),
    (dict(lda=63), None, INVALID), (dict(ldb=48), None, INVALID), (dict(ldd=63), None, INVALID),
    (dict(K=60, lda=60), None, MISALIGNED), (dict(ldb=72), None, MISALIGNED), (dict(A=P + 8), None, MISALIGNED),
    (dict(B=P + 1), None, MISALIGNED), (dict(D=P + 8), None, MISALIGNED), (dict(ldd=66), None, MISALIGNED),
    (dict(scale_a=P + 2), None, MISALIGNED), (dict(scale_b=P + 1), None, MISALIGNED),
    (dict(K=1 << 17, lda=1 << 17, ldb=1 << 17), None, UNSUPPORTED),  # a sum may pass 32 bits
    (dict(lda=1 << 31), None, UNSUPPORTED), (dict(ldb=FAR), None, UNSUPPORTED), (dict(ldd=FAR), None, UNSUPPORTED),
    (dict(lda=1 << 26), None, UNSUPPORTED),  # a tile's rows span 2^31 bytes
    (dict(M=2, K=4096, lda=4096, ldb=1 << 26), None, UNSUPPORTED),  # so do 64 of the kernel of few rows
    (dict(M=1 << 40), None, UNSUPPORTED), (dict(N=1 << 40, ldd=1 << 40), None, UNSUPPORTED),
    (dict(M=1 << 30, N=1 << 30, ldd=1 << 30), None, UNSUPPORTED),  # too many tiles
    (dict(), dict(act=5), INVALID), (dict(), dict(act=-1), INVALID), (dict(), dict(backward=2), INVALID),
    (dict(), dict(backward=1), UNSUPPORTED), (dict(), dict(bias=P, bias_type=3), INVALID),
    (dict(), dict(bias=P + 2), MISALIGNED), (dict(), dict(residual=P, ldr=63), INVALID),
    (dict(), dict(residual=P + 8, ldr=64), MISALIGNED), (dict(), dict(pre=P, ldp=60), INVALID),
    (dict(), dict(pre=P, ldp=65), MISALIGNED), (dict(), dict(residual=P, ldr=FAR), UNSUPPORTED),
    (dict(), dict(pre=P, ldp=1 << 26), UNSUPPORTED),
    (dict(tune=(8, 8, 8, 1, 4)), None, UNSUPPORTED), (dict(tune=(256, 256, 32, 2, 8, 32, 0, 4)), None, UNSUPPORTED),
    (dict(tune=(128, 128, 64, 4, 8, 16, 0, 4, 0, 256)), None, UNSUPPORTED),  # stream-K
    (dict(tune=(128, 128, 64, 4, 8, 16, 0, 4, 2, 256)), None, INVALID),
    (dict(tune=(128, 128, 64, 4, 8, 16, 0, 4, 0, -1)), None, INVALID),
    (dict(K=8192, lda=8192, ldb=8192, tune=(256, 256, 64, 2, 8, 16, 1, 4, 2, 0)), None, UNSUPPORTED),  # no parts of that tile
    (dict(K=8192, lda=8192, ldb=8192, tune=(64, 64, 64, 4, 8, 16, 0, 4, 4, 0), wsb=1024), None, INVALID),  # short workspace
    (dict(K=8192, lda=8192, ldb=8192, tune=(64, 64, 64, 4, 8, 16, 0, 4, 4, 0), ws=P + 16), None, INVALID),
    (dict(M=0), None, OK), (dict(N=0), None, OK),
])
def test_product_refusals(call, e, expect):
    a = {**PRODUCT, **call}
    tune, ws, wsb = a.pop("tune", None), a.pop("ws", P), a.pop("wsb", 1 << 30)
    assert igc.gemm_int8_ex(*a.values(), None if e is None else epi(**e), tune, workspace=ws, workspace_bytes=wsb,
                            stream=0) == expect
    if tune is None:
        assert igc.gemm_int8(*a.values(), None if e is None else epi(**e), stream=0) == expect


def test_product_workspaces_and_choices():
    for M, N, K in ((-1, 8, 8), (8, -1, 8), (8, 8, -1), (8, 8, 1 << 17), (1 << 40, 8, 8)):
        assert igc.igc_gemm_int8_workspace_bytes(M, N, K) == -1
        with pytest.raises(ValueError):
            igc.igc_gemm_int8_default_tune(M, N, K)
    assert igc.igc_gemm_int8_workspace_bytes(64, 64, 8192, (64, 64, 64, 4, 8, 16, 0, 4, 4, 0)) == 4 * 64 * 64 * 4
    assert igc.igc_gemm_int8_workspace_bytes(64, 64, 64, (8, 8, 8, 1, 4)) == -1
    assert igc.igc_gemm_int8_workspace_bytes(0, 64, 8192, (64, 64, 64, 4, 8, 16, 0, 4, 4, 0)) == 0
    sizes = (1, 2, 8, 16, 17, 32, 33, 64, 65, 128, 200, 500, 777, 1024, 2048, 4096, 8192, 30000)
    for M in sizes:
        for N in sizes:
            for K in (0, 1, 15, 64, 1001, 4096, 16384, 131071):
                t = igc.igc_gemm_int8_default_tune(M, N, K)  # raises for a kernel that is not compiled
                need = igc.igc_gemm_int8_workspace_bytes(M, N, K)
                assert (need > 0) == (t.k_splits > 1), (M, N, K, t.k_splits, need)


def test_products_too_large_for_a_grid():
    """Sizes whose product of tiles, or of partial sums, would not fit 64 bits are refused by the call and its queries."""
    big, cut = (1 << 40) - 1, (64, 64, 64, 4, 8, 16, 0, 4, 16, 0)
    for M, N, tune in ((big, big, None), (big, 64, None), (64, big, None), ((1 << 31) - 1, (1 << 31) - 16, None),
                       ((1 << 31) - 1, (1 << 31) - 16, cut), (1 << 20, 1 << 20, cut), (1, 1 << 30, None),
                       (512, 512, (256, 256, 64, 2, 8, 16, 1, 4, 2, 0))):
        assert igc.igc_gemm_int8_workspace_bytes(M, N, 8192, tune) == -1, (M, N)
        assert igc.gemm_int8_ex(M, N, 8192, P, 8192, P, P, 8192, P, P, -(-N // 16) * 16, 0, None, tune, workspace=P,
                                workspace_bytes=1 << 62, stream=0) == UNSUPPORTED, (M, N)
        if tune is None:
            with pytest.raises(ValueError):
                igc.igc_gemm_int8_default_tune(M, N, 8192)


NORM = dict(M=4, C=24, x=P, ldx=24, residual=P, ldr=24, h=P, ldh=24, gamma=P, param_type=0, eps=1e-6, y=P, ldy=32, last=P)
ROWS = [(dict(M=-1), INVALID), (dict(C=0), INVALID), (dict(C=-8), INVALID), (dict(param_type=3), INVALID),
        (dict(x=None), INVALID), (dict(ldx=23), INVALID), (dict(ldr=16), INVALID), (dict(ldh=8), INVALID),
        (dict(y=None), INVALID), (dict(ldy=16), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
        (dict(x=P + 8), MISALIGNED), (dict(residual=P + 2), MISALIGNED), (dict(h=P + 4), MISALIGNED),
        (dict(y=P + 8), MISALIGNED), (dict(ldx=28), MISALIGNED), (dict(ldr=25), MISALIGNED), (dict(ldh=30), MISALIGNED),
        (dict(ldy=36), MISALIGNED), (dict(gamma=P + 2), MISALIGNED), (dict(gamma=P + 1, param_type=1), MISALIGNED),
        (dict(last=P + 2), MISALIGNED), (dict(M=1 << 40), UNSUPPORTED), (dict(ldx=FAR), UNSUPPORTED),
        (dict(ldy=FAR), UNSUPPORTED), (dict(C=1 << 30, ldx=1 << 30, ldr=1 << 30, ldh=1 << 30, ldy=1 << 30), UNSUPPORTED),
        (dict(M=1 << 33), UNSUPPORTED), (dict(M=0), OK)]


@pytest.mark.parametrize("call,expect", ROWS)
def test_norm_refusals(call, expect):
    for name in ("rms_norm_bf16", "rms_norm_fp16", "rms_norm_int8_bf16", "rms_norm_int8_fp16"):
        assert getattr(igc, name)(*{**NORM, **call}.values(), stream=0) == expect, name
    assert igc.rms_norm_int8_bf16(*{**NORM, "last": None}.values(), stream=0) == INVALID
    assert igc.rms_norm_int8_bf16(*{**NORM, "ldy": 24}.values(), stream=0) == MISALIGNED  # 8 bits: multiples of 16


BACK = dict(M=4, C=24, h=P, ldh=24, gamma=P, param_type=0, rstd=P, dy=P, lddy=24, dh=P, lddh=24, dx=P, lddx=24, dgamma=P)


@pytest.mark.parametrize("call,expect", [
    (dict(M=-1), INVALID), (dict(C=0), INVALID), (dict(param_type=-1), INVALID), (dict(h=None), INVALID),
    (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(rstd=None), INVALID), (dict(ldh=16), INVALID),
    (dict(lddy=16), INVALID), (dict(lddh=16), INVALID), (dict(lddx=16), INVALID), (dict(h=P + 8), MISALIGNED),
    (dict(dy=P + 8), MISALIGNED), (dict(dh=P + 8), MISALIGNED), (dict(dx=P + 8), MISALIGNED), (dict(lddx=28), MISALIGNED),
    (dict(gamma=P + 2), MISALIGNED), (dict(dgamma=P + 1, param_type=1), MISALIGNED), (dict(rstd=P + 2), MISALIGNED),
    (dict(M=1 << 40), UNSUPPORTED), (dict(lddy=FAR), UNSUPPORTED),
    (dict(M=4000, ws=P, wsb=256), INVALID), (dict(M=4000, ws=P + 16, wsb=1 << 30), INVALID),
])
def test_norm_backward_refusals(call, expect):
    a = {**BACK, **call}
    ws, wsb = a.pop("ws", None), a.pop("wsb", 0)
    for name in ("rms_norm_backward_bf16", "rms_norm_backward_fp16"):
        assert getattr(igc, name + "_ex")(*a.values(), workspace=ws, workspace_bytes=wsb, stream=0) == expect
        if ws is None:
            assert getattr(igc, name)(*a.values(), stream=0) == expect
    assert igc.rms_norm_backward_bf16(*{**BACK, "M": 0, "dgamma": None}.values(), stream=0) == OK


def test_norm_backward_workspaces():
    need = igc.igc_rms_norm_backward_workspace_bytes
    assert need(-1, 8) == need(8, 0) == need(1 << 40, 8) == need(8, 1 << 30) == -1
    assert need(0, 1000) == need(1, 1000) == 0
    assert need(8192, 4096) % 256 == 0 and 0 < need(8192, 4096) <= 64 << 20


def test_norm_backward_too_large():
    wide = dict(C=1 << 27, ldh=1 << 27, lddy=1 << 27, lddh=1 << 27, lddx=1 << 27)
    for call in (wide, {**wide, "M": 0}, dict(M=1 << 30)):
        assert igc.rms_norm_backward_bf16(*{**BACK, **call}.values(), stream=0) == UNSUPPORTED, call
    need = igc.igc_rms_norm_backward_workspace_bytes
    assert need(4, 1 << 27) == need(0, 1 << 27) == need(1 << 30, 8) == -1


QUANT = dict(M=4, C=24, act="silu", x=P, ldx=24, gate=P, ldg=24, q=P, ldq=32, scale=P)


@pytest.mark.parametrize("call,expect", [
    (dict(M=-1), INVALID), (dict(C=0), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(x=None), INVALID),
    (dict(q=None), INVALID), (dict(scale=None), INVALID), (dict(ldx=16), INVALID), (dict(ldg=16), INVALID),
    (dict(ldq=16), INVALID), (dict(x=P + 8), MISALIGNED), (dict(gate=P + 8), MISALIGNED), (dict(q=P + 8), MISALIGNED),
    (dict(ldx=28), MISALIGNED), (dict(ldg=28), MISALIGNED), (dict(ldq=40), MISALIGNED), (dict(scale=P + 2), MISALIGNED),
    (dict(M=1 << 40), UNSUPPORTED), (dict(ldg=FAR), UNSUPPORTED), (dict(M=1 << 33), UNSUPPORTED), (dict(M=0), OK),
])
def test_rows_to_8_bits_refusals(call, expect):
    for name in ("quantize_rows_int8_bf16", "quantize_rows_int8_fp16"):
        assert getattr(igc, name)(*{**QUANT, **call}.values(), stream=0) == expect


def test_host_tensors_are_refused():
    x, q, s = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError):
        igc.quantize_rows_int8_bf16(4, 32, "none", x, 32, None, 0, P, 32, P, stream=0)
    with pytest.raises(ValueError):
        igc.rms_norm_bf16(4, 32, P, 32, None, 0, None, 0, None, 0, 1e-6, x, 32, stream=0)
    with pytest.raises(ValueError):
        igc.gemm_int8(4, 4, 32, q, 32, P, P, 32, P, P, 8, 0, stream=0)
    with pytest.raises(ValueError):
        igc.gemm_int8(4, 4, 32, P, 32, s, P, 32, P, P, 8, 0, stream=0)
    with pytest.raises(ValueError):
        igc.gemm_int8(4, 4, 32, P, 32, P, P, 32, P, P, 8, 0, igc.Epilogue(residual=x), stream=0)
