"""Products of 8-bit integers, the RMS norm to 16 and to 8 bits with its gradient, and activations rounded to 8 bits,
through the C ABI against their definitions in 64 bits: types, one row to several tiles, odd sizes and strides, sums at
the end of 32 bits, rows of zeros, infinities and NaN, padding that must not be read or written, in-place outputs,
graphs, streams, and all of them in turn as a feed-forward block has them.

What the kernels may be off by, beside half a step of the stored type:
  - a sum of n terms of fp32 in a tree of depth d: d * 2^-24 * sum of magnitudes.  A row's sums have, in a thread, eight
    terms for each vector that it holds (at most four, or C / 8192 of a long row), then at most 22 joins: DEPTH(C);
  - rstd: half of the relative error of the mean square, and one rounding each for the mean, eps, the square root and
    the reciprocal;
  - the product: the exact sum rounded to fp32, one rounding for each scale, the last with the bias;
  - 8 bits: a value lies within half of scale of what it is rounded to, and 127 times the relative error of value times
    reciprocal (4 roundings) more.
"""
import itertools

import pytest
import torch

import implicit_gemm_conv_amd as igc
from fused_util import (ACT_LIP, ACT_REL, ACTS, DT, U32, act64, assert_within, generator, half_step, normal, padded,
                        round8)
from gpu_util import say, synchronize

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    igc.lib()


def up16(n):
    return (n + 15) // 16 * 16


def int8s(g, rows, cols, extra=16, low=-127):
    """(view, storage): random 8-bit integers in rows of a 16-byte multiple, 99 in the padding."""
    buf = torch.full((rows, up16(cols) + extra), 99, dtype=torch.int8)
    buf[:, :cols] = torch.randint(low, 128, (rows, cols), generator=g, dtype=torch.int16).to(torch.int8)
    buf = buf.cuda()
    return buf[:, :cols], buf


# ---- the product ----------------------------------------------------------------------------------------------------


class Product:
    def __init__(self, M, N, K, out="bf16", act="none", bias="f32", residual="out", pre=None, scales=True, seed=0):
        g = generator(seed)
        self.dims, self.act, self.out = (M, N, K), act, DT[out]
        self.A, self.Abuf = int8s(g, M, K)
        self.B, self.Bbuf = int8s(g, N, K)
        self.sa = (0.01 + torch.rand(M, generator=g) * 0.03).cuda() if scales else None
        self.sb = ((0.01 + torch.rand(N, generator=g)) * 0.03 * max(K, 1) ** -0.5).cuda() if scales else None
        self.bias = normal(g, N, scale=0.5, dtype=DT[bias]).cuda() if bias else None
        self.ldd = round8(N) + 8
        res_t = self.out if residual == "out" else DT.get(residual)
        self.res = padded(normal(g, M, N, dtype=res_t), self.ldd)[0] if residual else None
        self.pre, self.pre_buf = padded(torch.full((M, N), float("nan"), dtype=DT[pre]), self.ldd, extra_rows=2) if pre \
            else (None, None)
        self.define()

    def define(self):
        M, N, K = self.dims
        s = self.A.double() @ self.B.double().t() if K else torch.zeros(M, N, dtype=torch.float64, device="cuda")
        p = s * (self.sa.double()[:, None] if self.sa is not None else 1) * (self.sb.double() if self.sb is not None else 1)
        z = p + self.bias.double() if self.bias is not None else p
        ez = 2.01 * U32 * p.abs() + U32 * (p.abs() + z.abs())
        y = act64(z, self.act)
        tol = ez * ACT_LIP + (ACT_REL * (1 + z * z) * y.abs() if self.act not in ("none", "relu") else 0)
        if self.res is not None:
            tol = tol + U32 * (y.abs() + self.res.double().abs())
            y = y + self.res.double()
        self.z, self.ez, self.y, self.tol = z, ez, y, tol

    def run(self, tune=None, workspace=None, D=None, residual=None, stream=None):
        M, N, K = self.dims
        if D is None:
            D = torch.full((M + 2, self.ldd), float("nan"), dtype=self.out, device="cuda")
        e = igc.Epilogue(act=self.act, bias=self.bias, residual=self.res if residual is None else residual, pre=self.pre,
                         ldr=self.ldd, ldp=self.ldd)
        igc.check(igc.gemm_int8_ex(M, N, K, self.Abuf, self.Abuf.stride(0), self.sa, self.Bbuf, self.Bbuf.stride(0),
                                   self.sb, D, self.ldd, igc.out_code(self.out), e, tune, workspace, stream=stream))
        return D

    def check(self, D, what=""):
        M, N, _ = self.dims
        synchronize()
        assert torch.isnan(D[:M, N:].float()).all() and torch.isnan(D[M:].float()).all(), f"{what}: stray store"
        assert_within(D[:M, :N], self.y, self.tol, what)
        if self.pre is not None:
            assert_within(self.pre, self.z, self.ez, what + " pre")
            assert torch.isnan(self.pre_buf[:M, N:].float()).all() and torch.isnan(self.pre_buf[M:].float()).all()


SIZES = [(1, 1, 1), (1, 24, 200), (3, 17, 33), (16, 130, 64), (17, 257, 129), (33, 40, 1000), (64, 300, 260),
         (65, 65, 65), (129, 127, 15), (200, 96, 16), (300, 520, 100), (31, 70, 17), (40, 33, 255)]
TILES = [c for c in igc.tunes(igc.SCOPE_EPILOGUE) if c in igc.tunes(igc.SCOPE_ALL)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_product_sizes(M, N, K, out):
    p = Product(M, N, K, out, act="silu", pre="f32" if M % 2 else None, seed=M)
    p.check(p.run(), f"{M}x{N}x{K} {out}")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [5, 40, 150])
def test_product_activations(act, M):
    p = Product(M, 136, 96, "bf16", act=act, bias="bf16", residual="f32", pre="bf16", seed=1)
    p.check(p.run(), f"{act} {M}")


@pytest.mark.parametrize("M", [1, 20, 70])
def test_product_parts_left_out(M):
    for bias, residual, scales in itertools.product((None, "f16"), (None, "bf16"), (False, True)):
        p = Product(M, 100, 72, "f32", bias=bias, residual=residual, scales=scales, seed=2)
        p.check(p.run(), f"{M} {bias} {residual} {scales}")
    p = Product(M, 100, 72, "f32", bias=None, residual=None, seed=2)
    D = torch.full((M + 2, p.ldd), float("nan"), device="cuda")
    igc.check(igc.gemm_int8(M, 100, 72, p.Abuf, p.Abuf.stride(0), p.sa, p.Bbuf, p.Bbuf.stride(0), p.sb, D, p.ldd,
                            igc.OUT_F32))  # no epilogue at all
    p.check(D, "plain")


@pytest.mark.parametrize("cfg", TILES, ids=str)
@pytest.mark.parametrize("K", [1, 16, 127, 128, 640, 1001])
def test_product_of_every_tile(cfg, K):
    bm, bn = cfg[:2]
    for M, N in ((bm, bn), (bm + 3, 2 * bn + 5)):
        p = Product(M, N, K, "bf16", act="gelu_tanh", seed=K)
        p.check(p.run(igc.tune(cfg)), f"{cfg} {M}x{N}x{K}")


@pytest.mark.parametrize("cfg", [c for c in TILES if c[0] * c[1] <= 256 * 128], ids=str)
@pytest.mark.parametrize("M,N,K,splits", [(70, 130, 4097, 3), (300, 131, 8200, 5), (33, 64, 2048, 16)])
def test_product_in_parts(cfg, M, N, K, splits):
    p = Product(M, N, K, "bf16", act="gelu", seed=5)
    tune = igc.tune(cfg, k_splits=splits)
    ws = torch.empty(igc.igc_gemm_int8_workspace_bytes(M, N, K, tune), dtype=torch.uint8, device="cuda")
    D = p.run(tune, ws)
    p.check(D, f"{cfg} in {splits}")
    # the sum is exact, so every schedule gives the same bits
    whole = p.run(igc.tune(cfg))
    synchronize()
    assert torch.equal(D[:M, :N], whole[:M, :N])


@pytest.mark.parametrize("M,N,K", [(1, 40, 30000), (5, 300, 12345), (8, 1000, 16400), (20, 24, 4000), (32, 500, 4095),
                                   (16, 130, 8191), (7, 12, 100003)])
def test_product_of_few_rows(M, N, K):
    t = igc.igc_gemm_int8_default_tune(M, N, K)
    assert t.bm == 0, "the kernel of few rows"
    p = Product(M, N, K, "bf16", act="silu", seed=6)
    p.check(p.run(), f"{M}x{N}x{K}")


def test_product_of_the_largest_sums():
    """Every term 2^14 or its negative, as many as are allowed: sums at both ends of 32 bits, exact to fp32's rounding."""
    K = (1 << 17) - 1
    B = torch.full((65, up16(K)), -128, dtype=torch.int8, device="cuda")
    for M in (2, 70):
        A = torch.full((M, up16(K)), -128, dtype=torch.int8, device="cuda")
        A[1] = 127
        for tune in (None, igc.tune(TILES[0]), igc.tune(TILES[1], k_splits=3)):
            D = torch.zeros(M, 68, device="cuda")
            igc.check(igc.gemm_int8_ex(M, 65, K, A, up16(K), None, B, up16(K), None, D, 68, igc.OUT_F32, None, tune))
            synchronize()
            assert (D[0, :65] == float(K << 14)).all() and (D[1, :65] == float(torch.tensor(-127 * 128 * K).float())).all()


def test_product_schedules_and_workspaces():
    for M, N, K in ((1, 4096, 4096), (17, 8192, 2048), (777, 1336, 1001), (2048, 1024, 16384), (8192, 8192, 8192), (1, 512, 100000)):
        t = igc.igc_gemm_int8_default_tune(M, N, K)
        need = igc.igc_gemm_int8_workspace_bytes(M, N, K)
        assert (need > 0) == (t.k_splits > 1)
        say(M, N, K, t.astuple(), t.k_splits, need)
    M, N, K = 500, 500, 16384
    need = igc.igc_gemm_int8_workspace_bytes(M, N, K)
    assert need > 0
    p = Product(M, N, K, "bf16", seed=7)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    before = igc.igc_pool_allocations()
    given = p.run(workspace=ws)
    assert igc.igc_pool_allocations() == before
    p.check(given)
    pooled = p.run()
    synchronize()
    assert igc.igc_pool_allocations() == before + 1 and torch.equal(pooled[:M, :N], given[:M, :N])
    with pytest.raises(igc.IgcError) as err:
        p.run(workspace=ws[:need - 256])
    assert err.value.status == igc.IGC_ERR_INVALID_VALUE


@pytest.mark.parametrize("M", [3, 90])
def test_product_in_place_residual_and_empty_sums(M):
    p = Product(M, 90, 64, "bf16", act="relu", seed=8)
    D = torch.full((M + 2, p.ldd), float("nan"), dtype=p.out, device="cuda")
    D[:M, :90] = p.res
    p.check(p.run(D=D, residual=D), "in place")
    p = Product(M, 90, 0, "f32", act="silu", seed=9)
    p.check(p.run(), "K = 0")
    assert igc.gemm_int8(0, 8, 8, None, 16, None, None, 16, None, None, 8, igc.OUT_F32) == igc.IGC_OK


@pytest.mark.parametrize("M", [4, 100])
def test_product_scales_that_are_not_numbers(M):
    p = Product(M, 70, 100, "f32", bias=None, residual=None, seed=10)
    p.sa[1], p.sb[5] = float("nan"), float("inf")
    D = p.run()
    synchronize()
    D = D[:M, :70]
    bad = torch.zeros(M, 70, dtype=torch.bool, device="cuda")
    bad[1], bad[:, 5] = True, True
    assert torch.isfinite(D[~bad]).all() and torch.isnan(D[1]).all()
    s = p.A.double() @ p.B.double()[5]
    col = torch.where(s == 0, torch.full_like(s, float("nan")), s.sign() * float("inf"))
    col[1] = float("nan")
    assert torch.equal(torch.nan_to_num(D[:, 5].double(), nan=7.0), torch.nan_to_num(col, nan=7.0))


def test_product_scales_at_odd_addresses():
    for M in (2, 70):
        p = Product(M, 90, 100, "bf16", bias="bf16", seed=11)
        for name, dt in (("sa", torch.float32), ("sb", torch.float32), ("bias", torch.bfloat16)):
            v = getattr(p, name)
            buf = torch.zeros(v.numel() + 1, dtype=dt, device="cuda")
            buf[1:] = v
            setattr(p, name, buf[1:])
        p.check(p.run(), str(M))


def test_product_long_leading_dimensions():
    """Operand rows so far apart that their offsets pass 32 bits, and within a tile nearly 31."""
    M, N, K, ld = 300, 300, 100, (1 << 24) - 1024
    small = Product(M, N, K, "bf16", seed=12)
    A, B = (torch.empty(M * ld, dtype=torch.int8, device="cuda").view(M, ld) for _ in range(2))  # 5 GB each
    A[:, :K], B[:, :K] = small.A, small.B
    A[:, K:K + 16], B[:, K:K + 16] = 99, 99
    small.Abuf, small.Bbuf = A, B
    for cfg in ((64, 64, 64, 4, 8, 16, 0, 4), (128, 128, 64, 4, 8, 16, 0, 4)):
        small.check(small.run(igc.tune(cfg)), f"{cfg}")
    assert igc.gemm_int8_ex(M, N, K, A, ld, None, B, ld, None, small.res, small.ldd, igc.OUT_BF16, None,
                            igc.tune((256, 256, 64, 2, 8, 16, 1, 4))) == igc.IGC_ERR_UNSUPPORTED


# ---- rows -----------------------------------------------------------------------------------------------------------


def DEPTH(C):
    return 8 * max(4, -(-C // 8192)) + 22


NORM = {"bf16": igc.rms_norm_bf16, "fp16": igc.rms_norm_fp16}
NORM8 = {"bf16": igc.rms_norm_int8_bf16, "fp16": igc.rms_norm_int8_fp16}
BACK = {"bf16": igc.rms_norm_backward_bf16_ex, "fp16": igc.rms_norm_backward_fp16_ex}
QUANT = {"bf16": igc.quantize_rows_int8_bf16, "fp16": igc.quantize_rows_int8_fp16}
EPS = 1e-6
# every number of threads and vectors of a row, for few rows and many, whole vectors and not, and long rows
WIDTHS = [1, 7, 8, 100, 128, 130, 511, 512, 1001, 1024, 2048, 2049, 4000, 4096, 5071, 8192, 16380, 16384, 20000, 32768,
          32769, 50001]


def check_int8(q, qbuf, scale, v, rel, what):
    """q and scale are what rows v (float64), known to `rel` of each value and of the largest, go to."""
    M, C = v.shape
    assert (qbuf[:M, C:] == 99).all() and (qbuf[M:] == 99).all(), f"{what}: stray store"
    top = v.abs().amax(1)
    want = top / 127
    rtop = rel.amax(1) if torch.is_tensor(rel) else rel
    off = (scale.double() - want).abs()
    assert (off <= want * (rtop + 4 * U32) + 2.0 ** -149).all(), f"{what}: scale off by {(off / want).max().item():.3g}"
    live = top > 0
    assert (q[~live] == 0).all()
    steps = v[live] / want[live][:, None]
    far = (q[live].double() - steps).abs()
    r = rel[live] + rtop[live][:, None] if torch.is_tensor(rel) else 2 * rel
    bound = 0.5 + steps.abs() * (r + 4 * U32)
    assert (far <= bound).all(), f"{what}: {(far - bound).max().item():.3g} beyond"
    assert (q[live].abs().amax(1) == 127).all(), what


class Norm:
    def __init__(self, M, C, dtype="bf16", residual=True, gamma="f32", seed=0, width=1.0):
        g, t = generator(seed), DT[dtype]
        self.M, self.C, self.dtype, self.t = M, C, dtype, t
        ld = self.ld = round8(C) + 8
        self.x, self.xbuf = padded(normal(g, M, C, scale=width, dtype=t), ld)
        self.res = padded(normal(g, M, C, scale=2 * width, dtype=t), ld)[0] if residual else None
        self.gamma = (1 + normal(g, C, scale=0.3)).to(DT[gamma]).cuda() if gamma else None
        self.dy, _ = padded(normal(g, M, C, dtype=t), ld)
        self.dh, _ = padded(normal(g, M, C, scale=0.5, dtype=t), ld)
        self.define()

    def define(self):
        self.h = self.x if self.res is None else (self.x.float() + self.res.float()).to(self.t)
        hd = self.h.double()
        self.g64 = self.gamma.double() if self.gamma is not None else torch.ones(self.C, dtype=torch.float64, device="cuda")
        self.rstd = 1 / torch.sqrt((hd * hd).mean(1) + EPS)
        self.rstd_rel = (0.5 * (DEPTH(self.C) + 2) + 3) * U32
        self.y = hd * self.rstd[:, None] * self.g64

    def out(self, dtype=None, extra=2):
        return torch.full((self.M + extra, self.ld), float("nan"), dtype=dtype or self.t, device="cuda")

    def args(self):
        p = igc.out_code(self.gamma.dtype) if self.gamma is not None else 0
        return (self.x, self.ld, self.res, self.ld), (self.gamma, p, EPS)

    def forward(self, y=None, h=None, rstd=None, stream=None):
        a, b = self.args()
        igc.check(NORM[self.dtype](self.M, self.C, *a, h, self.ld, *b, y, self.ld, rstd, stream=stream))

    def check(self, y, h=None, rstd=None, what=""):
        synchronize()
        M, C = self.M, self.C
        for o in (y, h):
            if o is not None:
                assert torch.isnan(o[:M, C:].float()).all() and torch.isnan(o[M:].float()).all(), f"{what}: stray store"
        assert_within(y[:M, :C], self.y, self.y.abs() * (self.rstd_rel + 2.01 * U32), what)
        if h is not None:
            assert torch.equal(h[:M, :C], self.h), f"{what}: h"
        if rstd is not None:
            assert_within(rstd, self.rstd, self.rstd * self.rstd_rel, what + " rstd")

    def backward(self, dx, dgamma=None, dh=True, workspace=None, rstd=None, h=None, dy=None, stream=None):
        h = self.padded_h() if h is None else h
        igc.check(BACK[self.dtype](self.M, self.C, h, self.ld, self.gamma,
                                   igc.out_code(self.gamma.dtype) if self.gamma is not None else 0,
                                   self.rstd.float() if rstd is None else rstd, self.dy if dy is None else dy, self.ld,
                                   self.dh if dh else None, self.ld, dx, self.ld, dgamma, workspace, stream=stream))

    def padded_h(self):
        buf = torch.full((self.M, self.ld), float("nan"), dtype=self.t, device="cuda")
        buf[:, :self.C] = self.h
        return buf

    def check_backward(self, dx, dgamma=None, dh=True, what=""):
        synchronize()
        M, C = self.M, self.C
        assert torch.isnan(dx[:M, C:].float()).all() and torch.isnan(dx[M:].float()).all(), f"{what}: stray store"
        hd, dy, rs = self.h.double(), self.dy.double(), self.rstd[:, None]
        g, xh = dy * self.g64, hd * rs
        mean = (g * xh).mean(1, keepdim=True)
        want = rs * (g - xh * mean)
        # rstd comes in fp32 (a relative 2^-24 wherever it stands); the sum; at most six roundings of either term
        tol = rs * ((xh * (g * xh).abs().mean(1, keepdim=True)).abs() * (DEPTH(C) + 12) + g.abs() * 6) * U32
        if dh:
            want = want + self.dh.double()
            tol = tol + U32 * (want.abs() + self.dh.double().abs())
        assert_within(dx[:M, :C], want, tol, what + " dx")
        if dgamma is not None:
            terms = dy * xh
            assert_within(dgamma, terms.sum(0), (M + 4) * U32 * terms.abs().sum(0), what + " dgamma")


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("M", [1, 5, 700])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_norm(M, C, dtype):
    if M == 700 and C > 20000:
        M = 40
    n = Norm(M, C, dtype, residual=C % 3 != 0, gamma=("f32", "bf16", "f16", None)[C % 4], seed=C)
    y, h, rstd = n.out(), n.out(), torch.empty(M, device="cuda")
    n.forward(y, h, rstd)
    n.check(y, h, rstd, f"{M}x{C}")


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("M", [1, 5, 700])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_norm_to_8_bits(M, C, dtype):
    if M == 700 and C > 20000:
        M = 40
    n = Norm(M, C, dtype, residual=C % 3 != 0, gamma=("f32", "bf16", "f16", None)[C % 4], seed=C + 1)
    h, scale = n.out(), torch.empty(M, device="cuda")
    qbuf = torch.full((M + 2, up16(C) + 16), 99, dtype=torch.int8, device="cuda")
    a, b = n.args()
    igc.check(NORM8[dtype](M, C, *a, h, n.ld, *b, qbuf, qbuf.stride(0), scale))
    synchronize()
    assert torch.equal(h[:M, :C], n.h) and torch.isnan(h[:M, C:].float()).all() and torch.isnan(h[M:].float()).all()
    check_int8(qbuf[:M, :C], qbuf, scale, n.y, n.rstd_rel + 2 * U32, f"{M}x{C}")


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("M", [1, 5, 700])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_norm_backward(M, C, dtype):
    if M == 700 and C > 20000:
        M = 300 if C > 40000 else 40
    n = Norm(M, C, dtype, residual=C % 3 != 0, gamma=("f32", "bf16", "f16", None)[C % 4], seed=C + 2)
    dgamma = torch.empty(C, dtype=n.gamma.dtype if n.gamma is not None else torch.float32, device="cuda")
    dx, dh = n.out(), C % 2 == 0
    n.backward(dx, dgamma, dh)
    n.check_backward(dx, dgamma, dh, f"{M}x{C}")


def test_norm_of_many_short_rows():
    """Several rows a workgroup, far more rows than workgroups."""
    for M, C in ((20011, 72), (9001, 300), (4099, 700)):
        n = Norm(M, C, seed=M)
        y, dx, dgamma = n.out(), n.out(), torch.empty(C, device="cuda")
        n.forward(y)
        n.check(y, what=f"{M}x{C}")
        n.backward(dx, dgamma)
        n.check_backward(dx, dgamma, what=f"{M}x{C}")


@pytest.mark.parametrize("M,C,act,gate", [(3, 40, "none", False), (300, 1000, "silu", True), (33, 5071, "gelu", False),
                                          (700, 2048, "gelu_tanh", True), (2, 16384, "relu", True),
                                          (9, 33000, "silu", False), (600, 4096, "none", True), (1, 1, "silu", True),
                                          (40, 9000, "gelu", True), (700, 128, "silu", True)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rows_to_8_bits(M, C, act, gate, dtype):
    g, t = generator(C), DT[dtype]
    ld = round8(2 * C if C % 8 == 0 else 2 * round8(C)) + 8
    both = torch.full((M, ld), float("nan"), dtype=t)  # x and gate beside each other
    at = round8(C)
    both[:, :C], both[:, at:at + C] = normal(g, M, C, scale=1.5, dtype=t), normal(g, M, C, dtype=t)
    both = both.cuda()
    x, u = both[:, :C], both[:, at:at + C]
    qbuf, scale = torch.full((M + 2, up16(C) + 16), 99, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    igc.check(QUANT[dtype](M, C, act, x, ld, u if gate else None, ld, qbuf, qbuf.stride(0), scale))
    synchronize()
    xd = x.double()
    v = act64(xd, act)
    rel = (ACT_REL * (1 + xd * xd) if act not in ("none", "relu") else torch.zeros_like(xd)) + 2 * U32
    check_int8(qbuf[:M, :C], qbuf, scale, v * u.double() if gate else v, rel, f"{M}x{C} {act}")


@pytest.mark.parametrize("C", [60, 1001, 40000])
def test_rows_that_are_not_ordinary(C):
    """Zeros, one value, tiny and huge values, infinities and NaN: each row alone, its neighbours untouched."""
    t, M = torch.bfloat16, 8
    x = normal(generator(C), M, C, dtype=t)
    x[0] = 0
    x[1] = 0
    x[1, C // 2] = -3
    x[2] *= 2.0 ** -126     # below what 127 / top can be held for
    x[3] *= 2.0 ** 50
    x[4, 7], x[5, C - 1] = float("inf"), float("nan")
    x, _ = padded(x, round8(C) + 8)
    ld = x.stride(0)
    qbuf, scale = torch.full((M, up16(C)), 99, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    igc.check(igc.quantize_rows_int8_bf16(M, C, "none", x, ld, None, 0, qbuf, up16(C), scale))
    synchronize()
    fine = [0, 1, 3, 6, 7]
    check_int8(qbuf[fine, :C], torch.full((1, up16(C)), 99), scale[fine], x[fine].double(), 2 * U32, "rows")
    assert scale[4] == float("inf") and torch.isnan(scale[5]) and (qbuf[4:6, :C] == 0).all()
    assert qbuf[1, C // 2] == -127 and scale[0] == 0
    # the tiny row: q as of any other, its scale to the lowest step
    d = x[2].double()
    steps = d / d.abs().max() * 127
    assert ((qbuf[2, :C].double() - steps).abs() <= 0.5 + 127 * 6 * U32).all()
    assert (scale[2].double() - d.abs().max() / 127).abs() <= 2.0 ** -149
    # the norm: rows 4 and 5 give NaN, a zero row zeros, the others what they are
    y, rstd = torch.empty(M, ld, dtype=t, device="cuda"), torch.empty(M, device="cuda")
    igc.check(igc.rms_norm_bf16(M, C, x, ld, None, 0, None, 0, None, 0, EPS, y, ld, rstd))
    igc.check(igc.rms_norm_int8_bf16(M, C, x, ld, None, 0, None, 0, None, 0, EPS, qbuf, up16(C), scale))
    synchronize()
    assert (y[0, :C] == 0).all() and scale[0] == 0 and (qbuf[0, :C] == 0).all()
    assert torch.isnan(y[4, 7]) and (y[4, :7] == 0).all() and rstd[4] == 0 and torch.isnan(scale[4])
    assert torch.isnan(y[5, :C]).all() and torch.isnan(rstd[5]) and torch.isnan(scale[5]) and (qbuf[4:6, :C] == 0).all()
    for m in (1, 3, 6, 7):
        d = x[m].double()
        want = d / torch.sqrt((d * d).mean() + EPS)
        assert_within(y[m, :C], want, want.abs() * ((DEPTH(C) + 2) / 2 + 6) * U32, f"row {m}")
    assert torch.isfinite(scale[[0, 1, 2, 3, 6, 7]]).all()


@pytest.mark.parametrize("C", [60, 40000])
def test_norm_without_eps(C):
    """eps 0: rows of zeros are NaN, as 0 / 0 is; the others are exact to the same bounds."""
    t, M = torch.bfloat16, 3
    x = normal(generator(C), M, C, dtype=t)
    x[1] = 0
    x, _ = padded(x, round8(C))
    ld = x.stride(0)
    y, rstd, scale = torch.empty(M, ld, dtype=t, device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    q = torch.full((M, up16(C)), 99, dtype=torch.int8, device="cuda")
    igc.check(igc.rms_norm_bf16(M, C, x, ld, None, 0, None, 0, None, 0, 0.0, y, ld, rstd))
    igc.check(igc.rms_norm_int8_bf16(M, C, x, ld, None, 0, None, 0, None, 0, 0.0, q, up16(C), scale))
    synchronize()
    assert rstd[1] == float("inf") and torch.isnan(y[1, :C]).all() and torch.isnan(scale[1]) and (q[1, :C] == 0).all()
    for m in (0, 2):
        d = x[m, :C].double()
        want = d / torch.sqrt((d * d).mean())
        assert_within(y[m, :C], want, want.abs() * ((DEPTH(C) + 2) / 2 + 6) * U32, f"row {m}")


def test_ties_go_to_even():
    C = 256
    x = torch.zeros(2, C, dtype=torch.bfloat16)
    x[0, 0] = 127  # scale 1: q is the value itself, halves to even
    x[0, 1:9] = torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 62.5, 63.5])
    x[1] = x[0] * 0.25
    q, s = torch.empty(2, C, dtype=torch.int8, device="cuda"), torch.empty(2, device="cuda")
    igc.check(igc.quantize_rows_int8_bf16(2, C, "none", x.cuda(), C, None, 0, q, C, s))
    synchronize()
    for m in range(2):
        assert q[m, :9].tolist() == [127, 0, 2, 2, 0, -2, -2, 62, 64] and s[m] == (1.0, 0.25)[m]


@pytest.mark.parametrize("C", [60, 1001, 4096, 40000])
def test_norm_in_place(C):
    n = Norm(9, C, residual=True, gamma="f16", seed=C)
    for h_is, y_is in (("x", "res"), ("res", "x"), (None, "x"), ("res", None)):
        bufs = {}
        for name in ("x", "res"):
            bufs[name] = n.out()
            bufs[name][:n.M, :C] = getattr(n, name)
        h = bufs[h_is] if h_is else n.out()
        y = bufs[y_is] if y_is else n.out()
        igc.check(igc.rms_norm_bf16(n.M, C, bufs["x"], n.ld, bufs["res"], n.ld, h, n.ld, n.gamma, igc.OUT_F16, EPS, y, n.ld))
        n.check(y, h, what=f"h in {h_is}, y in {y_is}")
    for name in ("dy", "dh", "h"):
        dx = n.out()
        dx[:n.M, :C] = getattr(n, name)
        dgamma, kept = torch.empty(C, dtype=torch.float16, device="cuda"), n.dh
        if name == "dh":
            n.dh = dx
        n.backward(dx, dgamma, h=dx if name == "h" else None, dy=dx if name == "dy" else None)
        n.dh = kept
        n.check_backward(dx, dgamma, what=f"dx in {name}")


def test_norm_backward_workspaces_and_empty():
    n = Norm(700, 1000, seed=3)
    need = igc.igc_rms_norm_backward_workspace_bytes(700, 1000)
    ws, before = torch.empty(need, dtype=torch.uint8, device="cuda"), igc.igc_pool_allocations()
    dx, dgamma = n.out(), torch.empty(1000, device="cuda")
    n.backward(dx, dgamma, workspace=ws)
    assert igc.igc_pool_allocations() == before
    n.check_backward(dx, dgamma)
    again, dgamma2 = n.out(), torch.empty(1000, device="cuda")
    n.backward(again, dgamma2)
    synchronize()
    assert igc.igc_pool_allocations() == before + 1
    assert torch.equal(dx[:700, :1000], again[:700, :1000]) and torch.equal(dgamma, dgamma2)
    n.backward(again)  # no dgamma: no workspace
    assert igc.igc_pool_allocations() == before + 1
    n.check_backward(again)
    with pytest.raises(igc.IgcError) as err:
        n.backward(dx, dgamma, workspace=ws[:need - 256])
    assert err.value.status == igc.IGC_ERR_INVALID_VALUE
    dgamma.fill_(5)
    igc.check(igc.rms_norm_backward_bf16(0, 1000, None, 1000, n.gamma, 0, None, None, 1000, None, 0, None, 1000, dgamma))
    synchronize()
    assert (dgamma == 0).all()


def test_norm_gradient_against_differences():
    """loss = sum(dy * y) + sum(dh * h): the library's gradients along random directions against central differences."""
    n = Norm(13, 200, "fp16", residual=True, seed=4)
    dx, dgamma = n.out(), torch.empty(200, device="cuda")
    n.backward(dx, dgamma)
    synchronize()
    hd, dy, dh = n.h.double(), n.dy.double(), n.dh.double()

    def loss(h, gamma):
        return (dy * h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * gamma).sum() + (dh * h).sum()

    step = 1e-5
    got = {"h": dx[:13, :200].double(), "gamma": dgamma.double()}
    at = {"h": hd, "gamma": n.g64}
    for name in at:
        v = torch.randn(at[name].shape, generator=generator(5), dtype=torch.float64).cuda()
        up, down = dict(at), dict(at)
        up[name], down[name] = at[name] + step * v, at[name] - step * v
        diff = (loss(*up.values()) - loss(*down.values())) / (2 * step)
        have = (got[name] * v).sum()
        half = half_step(got["h"], torch.float16) if name == "h" else 40 * U32 * (dy * hd).abs().sum(0)
        tol = ((half * 1.01 + 40 * U32 * got[name].abs()) * v.abs()).sum() + 1e-6 * diff.abs() + 1e-6
        assert (have - diff).abs() <= tol, (name, float(have), float(diff), float(tol))


def test_rows_far_apart():
    """Leading dimensions whose offsets pass 32 bits."""
    M, C, ld = 40, 72, (1 << 27)
    n = Norm(M, C, seed=6)
    big = [torch.empty(M * ld, dtype=torch.bfloat16, device="cuda").view(M, ld) for _ in range(3)]  # 10 GB each
    x, res, y = big
    x[:, :C], res[:, :C] = n.x, n.res
    q8 = torch.empty(M * ld, dtype=torch.int8, device="cuda").view(M, ld)
    s = torch.empty(M, device="cuda")
    igc.check(igc.rms_norm_bf16(M, C, x, ld, res, ld, x, ld, n.gamma, 0, EPS, y, ld))
    igc.check(igc.quantize_rows_int8_bf16(M, C, "none", y, ld, None, 0, q8, ld, s))
    synchronize()
    assert torch.equal(x[:, :C], n.h)
    assert_within(y[:, :C], n.y, n.y.abs() * (n.rstd_rel + 2.01 * U32), "y")
    check_int8(q8[:, :C], torch.full((1, C), 99), s, y[:, :C].double(), 2 * U32, "q")
    dgamma = torch.empty(C, device="cuda")
    res[:, :C], y[:, :C] = n.dh, n.dy
    igc.check(igc.rms_norm_backward_bf16(M, C, x, ld, n.gamma, 0, n.rstd.float(), y, ld, res, ld, y, ld, dgamma))
    synchronize()
    buf = n.out()
    buf[:M, :C] = y[:, :C]
    n.check_backward(buf, dgamma)


# ---- together -------------------------------------------------------------------------------------------------------


class Block:
    """A feed-forward block in 8 bits: norm, product, gated activation, product and the residual."""

    def __init__(self, M, D, F, dtype="bf16", seed=0):
        g, t = generator(seed), DT[dtype]
        self.dims, self.dtype, self.t = (M, D, F), dtype, t
        self.x, self.res = normal(g, M, round8(D), dtype=t).cuda(), normal(g, M, round8(D), scale=2.0, dtype=t).cuda()
        self.gamma = (1 + normal(g, D, scale=0.2)).to(t).cuda()
        self.w1, self.w1buf = int8s(g, 2 * F, D)
        self.w2, self.w2buf = int8s(g, D, F)
        self.s1 = (torch.rand(2 * F, generator=g) * 0.03 * D ** -0.5).cuda()
        self.s2 = (torch.rand(D, generator=g) * 0.03 * F ** -0.5).cuda()
        dev = dict(device="cuda")
        self.h, self.q1, self.c1 = torch.empty_like(self.x), torch.empty(M, up16(D), dtype=torch.int8, **dev), torch.empty(M, **dev)
        self.u = torch.empty(M, 2 * F, dtype=t, **dev)
        self.q2, self.c2 = torch.empty(M, up16(F), dtype=torch.int8, **dev), torch.empty(M, **dev)
        self.y = torch.empty_like(self.x)
        need = max(igc.igc_gemm_int8_workspace_bytes(M, 2 * F, D), igc.igc_gemm_int8_workspace_bytes(M, D, F), 256)
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def run(self, workspace=True):
        M, D, F = self.dims
        ld, code, ws = self.x.stride(0), igc.out_code(self.t), self.ws if workspace else None
        igc.check(NORM8[self.dtype](M, D, self.x, ld, self.res, ld, self.h, ld, self.gamma, code, EPS, self.q1, up16(D), self.c1))
        igc.check(igc.gemm_int8_ex(M, 2 * F, D, self.q1, up16(D), self.c1, self.w1buf, self.w1buf.stride(0), self.s1, self.u,
                                   2 * F, code, workspace=ws))
        igc.check(QUANT[self.dtype](M, F, "silu", self.u, 2 * F, self.u[:, F:], 2 * F, self.q2, up16(F), self.c2))
        igc.check(igc.gemm_int8_ex(M, D, F, self.q2, up16(F), self.c2, self.w2buf, self.w2buf.stride(0), self.s2, self.y, ld,
                                   code, igc.Epilogue(residual=self.h[:, :D]), workspace=ws))

    def check(self, what=""):
        """Each step from what the one before it stored."""
        synchronize()
        M, D, F = self.dims
        t = self.t
        h = (self.x.float() + self.res.float()).to(t)
        assert torch.equal(self.h[:, :D], h[:, :D]), what
        hd = h[:, :D].double()
        y = hd / torch.sqrt((hd * hd).mean(1, keepdim=True) + EPS) * self.gamma.double()
        none = torch.full((1, 16), 99)
        check_int8(self.q1[:, :D], none.new_full((1, D), 99), self.c1, y, ((DEPTH(D) + 2) / 2 + 5) * U32, what + " norm")
        p = (self.q1[:, :D].double() @ self.w1.double().t()) * self.c1.double()[:, None] * self.s1.double()
        assert_within(self.u, p, 4 * U32 * p.abs(), what + " up")
        a, b = self.u[:, :F].double(), self.u[:, F:].double()
        check_int8(self.q2[:, :F], none.new_full((1, F), 99), self.c2, act64(a, "silu") * b,
                   ACT_REL * (1 + a * a) + 2 * U32, what + " gate")
        p = (self.q2[:, :F].double() @ self.w2.double().t()) * self.c2.double()[:, None] * self.s2.double()
        assert_within(self.y[:, :D], p + hd, U32 * (5 * p.abs() + 2 * hd.abs()), what + " down")


@pytest.mark.parametrize("M,D,F,dtype", [(1, 520, 1040, "bf16"), (17, 1000, 264, "fp16"), (300, 257, 1032, "bf16"),
                                         (600, 512, 2048, "fp16")])
def test_feed_forward_block(M, D, F, dtype):
    b = Block(M, D, F, dtype, seed=M)
    b.run()
    b.check()


def test_captured_block_replays():
    """Blocks of one and of many tokens, the second with K splits, and a norm's gradient, captured and replayed on new
    inputs with eager work between; the graphs share one workspace and run one after the other."""
    blocks = [Block(1, 520, 1040, seed=1), Block(200, 512, 8192, seed=2)]
    blocks[0].ws = blocks[1].ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    n = Norm(700, 1000, seed=3)
    h, rstd, dx, dgamma = n.padded_h(), n.rstd.float(), n.out(), torch.empty(1000, device="cuda")
    graphs = []
    for f in (blocks[0].run, blocks[1].run, lambda: n.backward(dx, dgamma, workspace=blocks[0].ws, rstd=rstd, h=h)):
        f()
        synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f()
        graphs.append(graph)
    for turn in range(3):
        for b, graph in zip(blocks, graphs):
            g = generator(50 + turn)
            b.x.copy_(normal(g, *b.x.shape, dtype=b.t))
            for o in (b.h, b.u, b.y, b.c1, b.c2):
                o.fill_(float("nan"))
            graph.replay()
            b.check(f"replay {turn}")
            kept = b.y.clone()
            b.run(workspace=False)  # eager, from the pool
            b.check(f"eager {turn}")
            assert torch.equal(kept, b.y)
        n.dy.copy_(normal(generator(60 + turn), 700, 1000, dtype=n.t))
        dx.fill_(float("nan"))
        graphs[2].replay()
        n.check_backward(dx, dgamma, what=f"replay {turn}")


def test_pool_workspaces_are_refused_under_capture():
    p, n = Product(500, 500, 16384, "bf16", seed=7), Norm(700, 1000, seed=3)
    D, dx, dgamma = p.run(), n.out(), torch.empty(1000, device="cuda")
    rstd, h = n.rstd.float(), n.padded_h()
    synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for f in (lambda: p.run(D=D), lambda: n.backward(dx, dgamma, rstd=rstd, h=h)):
            with pytest.raises(igc.IgcError) as err:
                f()
            assert err.value.status == igc.IGC_ERR_UNSUPPORTED
        dx.zero_()


def test_streams_at_once():
    blocks = [Block(17, 1000, 264, "fp16", seed=1), Block(200, 512, 8192, seed=2)]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.run(workspace=False)
    torch.cuda.synchronize()
    for k, b in enumerate(blocks):
        b.check(f"stream {k}")


def test_pinned_tensors():
    x = normal(generator(1), 4, 64, dtype=torch.bfloat16).pin_memory()
    q, s = torch.empty(4, 64, dtype=torch.int8, pin_memory=True), torch.empty(4, pin_memory=True)
    igc.check(igc.quantize_rows_int8_bf16(4, 64, "none", x, 64, None, 0, q, 64, s))
    synchronize()
    check_int8(q, torch.full((1, 64), 99), s, x.double(), 2 * U32, "pinned")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,C", [(300, 8192), (40, 1001), (3, 40000)])
def test_every_tie_goes_to_even(M, C, dtype):
    """Products of two 16-bit values are exact in fp32, and under a largest one that 127 divides many lie half-way between
    two integers (127 over it is 3.2 here, which fp32 rounds): q is the nearest integer of the exact ratio, or at a tie the
    even one.

    The ratio is rounded to fp32 first, whose steps from 64 on are 2^-17: a value that is no tie may become one from half
    of that away, and those within 2^-17 are left out."""
    t = DT[dtype]
    g = generator(C + M)
    x, u = normal(g, M, C, dtype=t), normal(g, M, C, dtype=t)
    gamma = torch.where(normal(g, C) > 0, 1.0, -0.5).to(t)
    x[::2], u[::2] = (8 * x[::2]).round().clamp(-50, 50) * 5 / 32, gamma
    x[:, 5], u[:, 5], gamma[5] = 127 / 8, 2.5, 2.5  # the largest of a row: 127 * 5 / 16; odd multiples of 5 / 32 are ties
    x[1], u[1] = x[1] * 2.0 ** -9, u[1] * 2.0 ** -3
    x, _ = padded(x, round8(C))
    u, _ = padded(u, round8(C))
    gamma = gamma.cuda()
    q, scale = torch.full((M, up16(C)), 99, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")

    def check(v):
        steps = v * 127 / v.abs().amax(1, keepdim=True)
        beside = (steps - steps.floor() - 0.5).abs()
        ties = beside == 0
        assert ties.sum() >= C // 100, ties.sum()
        wrong = (q[:, :C].double() != steps.round()) & (ties | (beside > 2.0 ** -17))
        assert not wrong.any(), (wrong.nonzero()[:4], wrong.sum(), ties.sum())

    igc.check(QUANT[dtype](M, C, "none", x, x.stride(0), u, u.stride(0), q, up16(C), scale))
    synchronize()
    check(x[:, :C].double() * u[:, :C].double())
    q.fill_(99)
    igc.check(NORM8[dtype](M, C, x, x.stride(0), None, 0, None, 0, gamma, igc.out_code(t), EPS, q, up16(C), scale))
    synchronize()
    check(x[:, :C].double() * gamma.double())


OWN_TILES = [(64, 64, 64, 5, 8, 16, 0, 4), (32, 64, 64, 5, 4, 16, 0, 0)]


@pytest.mark.parametrize("cfg", OWN_TILES, ids=str)
@pytest.mark.parametrize("K", [1, 16, 127, 128, 640, 1001, 1300])
def test_product_of_its_own_tiles(cfg, K):
    bm, bn = cfg[:2]
    for M, N, act in ((bm, bn, "gelu_tanh"), (bm + 3, 2 * bn + 5, "silu"), (1, 7, "none"), (3 * bm, 9 * bn, "none")):
        p = Product(M, N, K, "bf16", act=act, seed=K)
        p.check(p.run(igc.tune(cfg)), f"{cfg} {M}x{N}x{K}")


@pytest.mark.parametrize("cfg", OWN_TILES, ids=str)
@pytest.mark.parametrize("M,N,K,splits", [(70, 130, 4097, 3), (300, 131, 8200, 5), (33, 64, 2048, 16)])
def test_product_in_parts_of_its_own_tiles(cfg, M, N, K, splits):
    test_product_in_parts(cfg, M, N, K, splits)


@pytest.mark.parametrize("C", [200, 40000])
def test_rows_of_every_magnitude(C):
    """A row times a power of two goes to the same integers, and its scale is that much larger, exactly."""
    row = normal(generator(C), 1, C, dtype=torch.bfloat16).clamp(-60, 60)
    row[0, ::3] = (4 * row[0, ::3]).round() / 4
    row[0, 5] = 127 / 2  # odd multiples of 1 / 4 are ties
    powers = [0, 110, 120, -60, -97, -101, -115]
    x = torch.cat([row.float() * 2.0 ** p for p in powers]).to(torch.bfloat16)
    x, _ = padded(x, round8(C))
    q, scale = torch.full((len(powers), up16(C)), 99, dtype=torch.int8, device="cuda"), torch.empty(len(powers), device="cuda")
    igc.check(igc.quantize_rows_int8_bf16(len(powers), C, "none", x, x.stride(0), None, 0, q, up16(C), scale))
    synchronize()
    for i, p in enumerate(powers):
        assert torch.equal(q[i, :C], q[0, :C]), f"2^{p}"
        assert scale[i].item() == scale[0].item() * 2.0 ** p, f"2^{p}"
