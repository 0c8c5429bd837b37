"""The fused operators' entry points on the CPU: they refuse bad arguments before anything is launched, size their
workspaces, and the binding marshals what it is given.  No GPU is used."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import implicit_gemm_conv_amd as igc

pytestmark = pytest.mark.skipif(not os.path.exists(igc.LIB_PATH), reason="libigc.so not built")

P = 1 << 20  # a 16-byte aligned address that is never dereferenced (validation fails first)
INVALID, MISALIGNED, UNSUPPORTED = igc.IGC_ERR_INVALID_VALUE, igc.IGC_ERR_MISALIGNED, igc.IGC_ERR_UNSUPPORTED


def epi(**kw):
    c = igc.CEpilogue()
    for k, v in kw.items():
        setattr(c, k, v)
    return c


GEMM_CALL = dict(M=64, N=64, K=64, A=P, lda=64, la=0, B=P, ldb=64, lb=0, D=P, ldd=64, d_type=0)


@pytest.mark.parametrize("call,e,expect", [
    (dict(), None, INVALID),
    (dict(), dict(act=5), INVALID), (dict(), dict(act=-1), INVALID),
    (dict(), dict(backward=2), INVALID), (dict(), dict(backward=1, act=igc.ACT_SILU), INVALID),  # no pre to read
    (dict(), dict(bias=P, bias_type=3), INVALID), (dict(), dict(bias=P + 2), MISALIGNED),
    (dict(), dict(bias=P + 1, bias_type=1), MISALIGNED),
    (dict(), dict(residual=P, ldr=63), INVALID), (dict(), dict(residual=P, ldr=64, residual_type=-1), INVALID),
    (dict(), dict(residual=P + 8, ldr=64), MISALIGNED), (dict(), dict(residual=P, ldr=68, residual_type=1), MISALIGNED),
    (dict(), dict(pre=P, ldp=60), INVALID), (dict(), dict(pre=P, ldp=65), MISALIGNED),
    (dict(), dict(pre=P + 4, ldp=64), MISALIGNED), (dict(), dict(pre=P, ldp=64, pre_type=7), INVALID),
    (dict(M=-1), dict(), INVALID), (dict(d_type=4), dict(), INVALID), (dict(la=2), dict(), INVALID),
    (dict(ldd=63), dict(), INVALID), (dict(A=None), dict(), INVALID), (dict(A=P + 2), dict(), MISALIGNED),
    (dict(D=P + 8), dict(), MISALIGNED), (dict(M=65, tune=(256, 256, 32, 2, 8, 32, 0, 4)), dict(), UNSUPPORTED),
    (dict(M=512, K=8192, lda=8192, tune=(128, 128, 64, 4, 8, 16, 0, 4, 0, 16)), dict(), UNSUPPORTED),  # stream-K
    (dict(tune=(8, 8, 8, 1, 4)), dict(), UNSUPPORTED),
])
@pytest.mark.parametrize("name", ["gemm_bf16_epilogue_ex", "gemm_fp16_epilogue_ex"])
def test_gemm_epilogue_refusals(name, call, e, expect):
    a = {**GEMM_CALL, **call}
    tune = a.pop("tune", None)
    got = getattr(igc, name)(*a.values(), None if e is None else epi(**e), tune, workspace=P, workspace_bytes=1 << 30,
                             stream=0)
    assert got == expect


CONV_CALL = dict(N=1, H=8, W=8, C=16, K=16, R=3, S=3, sh=1, sw=1, ph=1, pw=1, dh=1, dw=1, x=P, w=P, y=P, y_type=1)


@pytest.mark.parametrize("call,e,expect", [
    (dict(), None, INVALID), (dict(), dict(act=9), INVALID), (dict(), dict(backward=1), UNSUPPORTED),
    (dict(), dict(residual=P + 2, residual_type=1), MISALIGNED), (dict(), dict(pre=P, pre_type=5), INVALID),
    (dict(C=12), dict(), MISALIGNED), (dict(x=None), dict(), INVALID), (dict(y=None), dict(), INVALID),
    (dict(R=9, ph=0), dict(), INVALID), (dict(y_type=-1), dict(), INVALID), (dict(x=P + 4), dict(), MISALIGNED),
])
def test_conv_epilogue_refusals(call, e, expect):
    a = {**CONV_CALL, **call}
    for name in ("conv2d_nhwc_implicit_gemm_epilogue", "conv2d_nhwc_implicit_gemm_epilogue_fp16"):
        assert getattr(igc, name)(*a.values(), None if e is None else epi(**e), stream=0) == expect


BACK_CALL = dict(M=4, N=24, act="silu", dD=P, ldd=24, pre=P, ldp=24, dz=P, ldz=24, dbias=P, dbias_type=0)


@pytest.mark.parametrize("call,expect", [
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(act=7), INVALID), (dict(dbias_type=3), INVALID),
    (dict(dz=None, dbias=None), INVALID), (dict(dD=None), INVALID), (dict(pre=None), INVALID), (dict(ldd=23), INVALID),
    (dict(ldp=16), INVALID), (dict(ldz=16), INVALID), (dict(dD=P + 2), MISALIGNED), (dict(ldd=28), MISALIGNED),
    (dict(ldp=25), MISALIGNED), (dict(dz=P + 8), MISALIGNED), (dict(dbias=P + 2), MISALIGNED),
    (dict(M=100000, workspace=P, workspace_bytes=256), INVALID), (dict(M=100000, workspace=P + 16, workspace_bytes=1 << 30), INVALID),
])
def test_epilogue_backward_refusals(call, expect):
    a = {**BACK_CALL, **call}
    ws, wsb = a.pop("workspace", None), a.pop("workspace_bytes", None)
    for name in ("epilogue_backward_bf16_ex", "epilogue_backward_fp16_ex"):
        assert getattr(igc, name)(*a.values(), workspace=ws, workspace_bytes=wsb or 0, stream=0) == expect
    assert igc.epilogue_backward_bf16(0, 8, "none", None, 8, None, 8, None, 8, None, 0, stream=0) == igc.IGC_OK
    assert igc.epilogue_backward_bf16(8, 0, "none", None, 8, None, 8, None, 8, None, 0, stream=0) == igc.IGC_OK


NORM_CALL = dict(N=2, H=4, W=4, C=32, G=4, x=P, ldx=32, gamma=P, beta=P, param_type=0, eps=1e-5, act="silu", y=P, ldy=32,
                 mean=P, rstd=P)
NORM_BACK = dict(N=2, H=4, W=4, C=32, G=4, x=P, ldx=32, gamma=P, beta=P, param_type=0, mean=P, rstd=P, act="silu", dy=P,
                 lddy=32, dx=P, lddx=32, dgamma=P, dbeta=P)
SHARED = [(dict(N=-1), INVALID), (dict(H=0), INVALID), (dict(C=0), INVALID), (dict(G=0), INVALID), (dict(G=5), INVALID),
          (dict(C=36, G=4, ldx=40), MISALIGNED), (dict(param_type=3), INVALID), (dict(act=5), INVALID),
          (dict(x=None), INVALID), (dict(x=P + 8), MISALIGNED), (dict(ldx=24), INVALID), (dict(ldx=36), MISALIGNED),
          (dict(gamma=P + 2), MISALIGNED), (dict(beta=P + 1, param_type=1), MISALIGNED), (dict(mean=P + 2), MISALIGNED),
          (dict(H=1 << 16, W=1 << 15), UNSUPPORTED), (dict(N=1 << 26), UNSUPPORTED)]


@pytest.mark.parametrize("call,expect", SHARED + [(dict(y=None), INVALID), (dict(ldy=31), INVALID), (dict(eps=-1.0), INVALID),
                                                  (dict(eps=float("nan")), INVALID), (dict(y=P + 4), MISALIGNED)])
def test_group_norm_refusals(call, expect):
    for name in ("group_norm_nhwc_bf16", "group_norm_nhwc_fp16"):
        assert getattr(igc, name)(*{**NORM_CALL, **call}.values(), stream=0) == expect
    assert igc.group_norm_nhwc_bf16(*{**NORM_CALL, "N": 0}.values(), stream=0) == igc.IGC_OK


@pytest.mark.parametrize("call,expect", SHARED + [(dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(mean=None), INVALID),
                                                  (dict(rstd=None), INVALID), (dict(lddy=16), INVALID), (dict(lddx=44), MISALIGNED),
                                                  (dict(dgamma=P + 2), MISALIGNED), (dict(dbeta=P + 2), MISALIGNED)])
def test_group_norm_backward_refusals(call, expect):
    for name in ("group_norm_nhwc_backward_bf16", "group_norm_nhwc_backward_fp16"):
        assert getattr(igc, name)(*{**NORM_BACK, **call}.values(), stream=0) == expect
    none = {**NORM_BACK, "N": 0, "dgamma": None, "dbeta": None}
    assert igc.group_norm_nhwc_backward_bf16(*none.values(), stream=0) == igc.IGC_OK


def test_workspace_sizes():
    assert igc.igc_epilogue_workspace_bytes(igc.OP_GEMM, 8192, 8192, 8192) == 0
    assert igc.igc_epilogue_workspace_bytes(igc.OP_GEMM, -1, 8, 8) == -1
    assert igc.igc_epilogue_workspace_bytes(igc.OP_CONV_WGRAD, 8, 8, 8) == -1
    assert igc.igc_epilogue_workspace_bytes(igc.OP_GEMM, 0, 8, 8) == 0
    # shapes that the plain product gives to stream-K split K here
    t = igc.igc_default_tune(1000, 512, 8192)
    assert t.stream_k > 0 and igc.igc_epilogue_workspace_bytes(igc.OP_GEMM, 1000, 512, 8192) >= 2 * 1000 * 512 * 4
    assert igc.igc_epilogue_backward_workspace_bytes(1, 100) == 0 and igc.igc_epilogue_backward_workspace_bytes(-1, 1) == -1
    assert igc.igc_epilogue_backward_workspace_bytes(1 << 20, 128) > 0
    assert igc.igc_group_norm_workspace_bytes(0, 4, 4, 32, 4) == 0
    assert igc.igc_group_norm_workspace_bytes(1, 4, 4, 32, 5) == -1
    assert igc.igc_group_norm_workspace_bytes(32, 256, 256, 256, 32) > 0


def test_every_shape_has_a_built_schedule():
    """The built-in choice names a configuration that the epilogue is built for, or a K split."""
    built = igc.tunes(igc.SCOPE_EPILOGUE)
    for op in (igc.OP_GEMM, igc.OP_CONV_FPROP):
        for M in (65, 100, 256, 1000, 4096, 100352):
            for N in (1, 64, 72, 256, 1000, 8192):
                for K in (0, 8, 72, 1000, 4096, 65536):
                    assert igc.igc_epilogue_workspace_bytes(op, M, N, K) >= 0
                    t = igc.igc_default_tune(M, N, K, op)
                    if t.stream_k == 0 and t.k_splits <= 1:
                        assert t.astuple() in built, (op, M, N, K, t.astuple())


def test_binding():
    t = torch.zeros(4, 24, dtype=torch.bfloat16)
    e = igc.Epilogue(act="gelu", bias=torch.zeros(24), residual=t, pre=t[:, :16].to(torch.float16), backward=True)
    assert (e.c.act, e.c.backward, e.c.bias_type, e.c.residual_type, e.c.ldr, e.c.pre_type, e.c.ldp) == (2, 1, 0, 1, 24, 2, 16)
    assert e.c.residual == t.data_ptr()
    assert igc.Epilogue(residual=t[:, :8]).c.ldr == 24
    assert igc.Epilogue().c.bias is None and igc.act_code(3) == 3
    with pytest.raises(ValueError):
        igc.Epilogue(residual=t.t())
    with pytest.raises(TypeError):
        igc.Epilogue(residual=P)
    with pytest.raises(TypeError):
        igc.out_code(torch.int8)
    with pytest.raises(KeyError):
        igc.Epilogue(act="tanh")
    assert igc.Epilogue(residual=P, ldr=8, residual_type=1).c.ldr == 8
    assert ctypes.sizeof(igc.CEpilogue) == 72 and len(e.raw) == 72
    assert bytes(e.c) == e.raw


def test_host_tensors_are_refused():
    """Every call refuses a tensor in host memory, in each of its places, and an epilogue that holds one, before the
    library is entered; what holds no values and plain addresses pass."""
    t, v = torch.zeros(64, 64, dtype=torch.bfloat16), torch.zeros(64)
    gemm, conv = dict(GEMM_CALL, N=16, ldd=16), CONV_CALL
    calls = [(igc.gemm_bf16, gemm, "ABD", ()), (igc.gemm_bf16_ex, gemm, "ABD", (None,)), (igc.gemm_bf16_noalloc, gemm, "ABD", ()),
             (igc.conv2d_nhwc_implicit_gemm, conv, "xwy", ()), (igc.conv2d_nhwc_wgrad_implicit_gemm_ex, conv, "xwy", (None,)),
             (igc.gemm_bf16_epilogue, gemm, "ABD", (epi(),)), (igc.gemm_fp16_epilogue_ex, gemm, "ABD", (epi(), None)),
             (igc.conv2d_nhwc_implicit_gemm_epilogue, conv, "xwy", (epi(),)),
             (igc.epilogue_backward_bf16, BACK_CALL, ("dD", "pre", "dz", "dbias"), ()),
             (igc.epilogue_backward_fp16_ex, BACK_CALL, ("dD", "pre", "dz", "dbias"), ()),
             (igc.group_norm_nhwc_bf16, NORM_CALL, ("x", "gamma", "beta", "y", "mean", "rstd"), ()),
             (igc.group_norm_nhwc_fp16_ex, NORM_CALL, ("x", "gamma", "beta", "y", "mean", "rstd"), ()),
             (igc.group_norm_nhwc_backward_bf16, NORM_BACK, ("x", "gamma", "beta", "mean", "rstd", "dy", "dx", "dgamma", "dbeta"), ())]
    for f, args, names, more in calls:
        for name in names:
            with pytest.raises(ValueError, match="host memory"):
                f(*{**args, name: t}.values(), *more, stream=0)
    with pytest.raises(ValueError, match="host memory"):
        igc.gemm_bf16_ex(*gemm.values(), None, torch.zeros(256, dtype=torch.uint8), stream=0)
    for parts in (dict(bias=v), dict(residual=t), dict(pre=t)):
        e = igc.Epilogue(**parts)  # the structure itself is made
        with pytest.raises(ValueError, match="host memory"):
            igc.gemm_bf16_epilogue(*gemm.values(), e, stream=0)
        with pytest.raises(ValueError, match="host memory"):
            igc.conv2d_nhwc_implicit_gemm_epilogue_ex(*conv.values(), e, stream=0)
    none = torch.empty(0)
    assert igc.gemm_bf16_epilogue(*{**gemm, "M": 0, "A": none, "D": none}.values(), epi(), stream=0) == igc.IGC_OK
    assert igc.gemm_bf16_epilogue(*{**gemm, "M": 0}.values(), igc.Epilogue(residual=P, ldr=64, residual_type=1), stream=0) == igc.IGC_OK


def test_workspace_queries_of_impossible_sizes():
    """The queries answer for any sizes, those that no call takes included (in a process of its own: a division by a
    block count cut to 32 bits ended it)."""
    code = """if True:
        import implicit_gemm_conv_amd as igc
        for k in (31, 32, 39, 40, 41, 47, 62):
            for d in (-257, -1, 0, 1):
                big = (1 << k) + d
                assert igc.igc_epilogue_backward_workspace_bytes(1000, big) == (-1 if big >= 1 << 31 else 0), big
                assert (igc.igc_epilogue_backward_workspace_bytes(big, 8) == -1) == (big >= 1 << 40), big
                for op in (igc.OP_GEMM, igc.OP_CONV_FPROP):
                    for sizes in ((big, 8, 8), (8, big, 8), (8, 8, big), (1, big, 4096), (big, 8, 4096)):
                        igc.igc_epilogue_workspace_bytes(op, *sizes)
        for sizes in ((2**31 - 1, 1, 1, 8, 1), (1, 2**31 - 1, 2**31 - 1, 8, 1), (1, 1, 1, 2**31 - 8, 1), (1, 46340, 46341, 8, 8)):
            assert igc.igc_group_norm_workspace_bytes(*sizes) >= -1
    """
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    for f in (igc.epilogue_backward_bf16, igc.epilogue_backward_fp16):
        assert f(*{**BACK_CALL, "N": 1 << 31, "ldd": 1 << 31, "ldp": 1 << 31, "ldz": 1 << 31}.values(), stream=0) == UNSUPPORTED
        assert f(*{**BACK_CALL, "M": 1 << 40}.values(), stream=0) == UNSUPPORTED


def test_launches_of_too_many_threads_are_refused():
    """Nothing is enqueued where one of a call's launches would have 2^32 threads: the sums of dgamma and dbeta would
    otherwise run after a launch that failed."""
    many, wide = dict(N=1 << 26, H=1, W=1, C=8, G=1, ldx=8), dict(N=1, H=1, W=1, C=1 << 28, G=1 << 25, ldx=1 << 28)
    for name in ("group_norm_nhwc_bf16", "group_norm_nhwc_fp16"):
        assert getattr(igc, name)(*{**NORM_CALL, **many, "ldy": 8}.values(), stream=0) == UNSUPPORTED
    for name in ("group_norm_nhwc_backward_bf16", "group_norm_nhwc_backward_fp16"):
        assert getattr(igc, name)(*{**NORM_BACK, **many, "lddy": 8, "lddx": 8}.values(), stream=0) == UNSUPPORTED
        for N in (0, 1):
            assert getattr(igc, name)(*{**NORM_BACK, **wide, "N": N, "lddy": 1 << 28, "lddx": 1 << 28}.values(), stream=0) == UNSUPPORTED


def test_a_convolution_takes_no_tensor_with_gaps():
    """A convolution reads and writes its residual and pre as dense NPQK: a slice of a wider tensor is refused, where its
    strides would be passed over.  A product takes such rows with their leading dimension."""
    wide = torch.zeros(1, 8, 8, 24, dtype=torch.bfloat16)
    rows = wide.reshape(64, 24)
    for name in ("residual", "pre"):
        for gaps in (wide[..., :16], wide[:, :, ::2], wide[:, 1:7, 1:]):
            with pytest.raises(ValueError, match="dense"):
                igc.Epilogue(**{name: gaps})
        for e in (igc.Epilogue(**{name: rows[:, :16]}), igc.Epilogue(**{name: wide[..., :16]}, ldr=24, ldp=24)):
            assert (e.c.ldr if name == "residual" else e.c.ldp) == 24
            for call, more in ((igc.conv2d_nhwc_implicit_gemm_epilogue, ()), (igc.conv2d_nhwc_implicit_gemm_epilogue_fp16_ex, (None,))):
                with pytest.raises(ValueError, match="dense"):
                    call(*CONV_CALL.values(), e, *more, stream=0)
        for dense in (wide, rows, wide[:, :, :, 8:9].contiguous(), wide[:, 2:6]):
            e = igc.Epilogue(**{name: dense})
            with pytest.raises(ValueError, match="host memory"):  # past the check above
                igc.conv2d_nhwc_implicit_gemm_epilogue(*CONV_CALL.values(), e, stream=0)


def test_the_fused_calls_choice_is_compiled():
    """The choice of calls with an epilogue, in every operand layout: its kernels are compiled for both types, it never is
    stream-K, the workspace query has room for its parts, and the sizes below reach every tile that it can name."""
    seen = set()
    full = igc.tunes(igc.SCOPE_EPILOGUE | igc.SCOPE_ALL)
    layouts = [(a, b) for a in (igc.ROW_MAJOR, igc.COL_MAJOR) for b in (igc.ROW_MAJOR, igc.COL_MAJOR)]
    sizes = [(M, N, K) for M in (1, 8, 9, 20, 21, 33, 65, 100, 200, 256, 1000, 2100, 4096, 100352)
             for N in (1, 64, 72, 256, 304, 1000, 2100, 8192, 16400, 33000) for K in (0, 8, 72, 520, 1000, 2085, 4096, 8192, 65536)]
    sizes += [(3000, 3000, 1000), (1536, 4096, 4096), (6000, 800, 800), (100352, 256, 2304), (22176, 304, 160), (12032, 72, 192)]
    for op in (igc.OP_GEMM, igc.OP_CONV_FPROP):
        for M, N, K in sizes:
            for la, lb in layouts if op == igc.OP_GEMM else layouts[:1]:
                t = igc.igc_epilogue_default_tune(M, N, K, op, la, lb)  # raises where it is not compiled
                need = igc.igc_epilogue_workspace_bytes(op, M, N, K)
                if t.k_splits > 1:  # (a ring period is at most 512 of K: fewer parts may be enough)
                    assert t.k_splits <= 256 and need >= 2 * M * N * 4, (op, M, N, K, la, lb)
                if t.bm == 0:
                    assert op == igc.OP_GEMM and la == igc.ROW_MAJOR and M <= 32 and t.bn in (16, 32, 64, 128)
                else:
                    assert t.stream_k == 0 and t.astuple() in (full if op == igc.OP_GEMM else igc.tunes(igc.SCOPE_EPILOGUE))
                seen.add((op, t.bm, t.bn, t.k_splits > 1))
    G, F = igc.OP_GEMM, igc.OP_CONV_FPROP
    assert seen >= {(G, 0, 16, False), (G, 0, 16, True), (G, 0, 32, False), (G, 0, 64, False), (G, 0, 128, False),
                    (G, 64, 64, False), (G, 64, 64, True), (G, 64, 128, False), (G, 64, 128, True), (G, 128, 128, False),
                    (G, 256, 128, False), (G, 256, 128, True), (G, 256, 256, False), (F, 64, 64, False), (F, 64, 128, False),
                    (F, 128, 64, False), (F, 256, 64, False), (F, 224, 256, False), (F, 256, 256, False)}, sorted(seen)
    for bad in ((igc.OP_CONV_WGRAD, 0, 0), (igc.OP_GEMM, 2, 0), (igc.OP_GEMM, 0, -1)):
        with pytest.raises(ValueError):
            igc.igc_epilogue_default_tune(64, 64, 64, *bad)
    with pytest.raises(ValueError):
        igc.igc_epilogue_default_tune(-1, 64, 64)
