"""Products and convolutions with a fused epilogue, and the epilogue's gradient, through the C ABI against their
definitions in 64 bits: types, operand layouts, one row to several tiles, odd sizes and leading dimensions, K from 0,
every activation in both directions, split K, in-place residuals, graphs and refusals that need a GPU."""
import itertools

import pytest
import torch

import implicit_gemm_conv_amd as igc
from fused_util import (ACT_CURVE, ACT_LIP, ACT_REL, ACTS, DT, GRAD_ABS, U32, act64, act_grad64, assert_within,
                        generator, half_step, normal, padded, round8)
from gpu_util import say, synchronize

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    igc.lib()


GEMM = {"bf16": igc.gemm_bf16_epilogue_ex, "fp16": igc.gemm_fp16_epilogue_ex}
BACK = {"bf16": igc.epilogue_backward_bf16_ex, "fp16": igc.epilogue_backward_fp16_ex}


class Problem:
    """Operands on the GPU with NaN in every padding element, and the expected results."""

    def __init__(self, M, N, K, dtype="bf16", out=None, la="row", lb="col", act="none", bias="f32", residual="in",
                 pre=None, backward=False, seed=0, pad=8):
        g, t = generator(seed), DT[dtype]
        self.dims, self.dtype, self.la, self.lb, self.act, self.backward = (M, N, K), dtype, la, lb, act, backward
        self.out = DT[out or dtype]
        A = normal(g, M, K, dtype=t)
        B = normal(g, N, K, scale=max(K, 1) ** -0.5, dtype=t)
        self.A, self.Abuf = padded(A if la == "row" else A.t(), round8(K if la == "row" else M) + pad)
        self.B, self.Bbuf = padded(B if lb == "col" else B.t(), round8(K if lb == "col" else N) + pad)
        self.bias = normal(g, N, scale=0.5, dtype=DT[bias]).cuda() if bias else None
        self.ldd = round8(N) + pad
        res_t = t if residual == "in" else DT.get(residual)
        self.res = padded(normal(g, M, N, dtype=res_t), self.ldd)[0] if residual else None
        pre_t = t if pre == "in" else DT.get(pre)
        self.pre_buf = None
        if backward and act != "none":
            self.pre, self.pre_buf = padded(normal(g, M, N, scale=2.0, dtype=pre_t or t), self.ldd)
        elif pre:
            self.pre, self.pre_buf = padded(torch.full((M, N), float("nan"), dtype=pre_t), self.ldd, extra_rows=2)
        else:
            self.pre = None
        # the definitions
        a, b = A.cuda().double(), B.cuda().double()
        z = a @ b.t() if K else torch.zeros(M, N, dtype=torch.float64, device="cuda")
        S = a.abs() @ b.abs().t() if K else torch.zeros_like(z)
        if bias:
            z, S = z + self.bias.double(), S + self.bias.double().abs()
        ez = (K + 2) * U32 * S
        if backward:
            p = self.pre.double() if self.pre is not None else torch.zeros_like(z)
            d = act_grad64(p, act)
            y, tol = z * d, ez * ACT_LIP + z.abs() * (GRAD_ABS if act != "none" else 0) + U32 * z.abs()
        else:
            y = act64(z, act)
            tol = ez * ACT_LIP + (ACT_REL * (1 + z * z) * y.abs() if act not in ("none", "relu") else 0)
        if residual:
            tol = tol + U32 * (y.abs() + self.res.double().abs())
            y = y + self.res.double()
        self.z, self.ez, self.y, self.tol = z, ez, y, tol

    def epilogue(self, residual=None):
        return igc.Epilogue(act=self.act, bias=self.bias, residual=self.res if residual is None else residual,
                            pre=self.pre, backward=self.backward, ldr=self.ldd, ldp=self.ldd)

    def run(self, tune=None, workspace=None, D=None, epilogue=None, stream=None):
        M, N, K = self.dims
        if D is None:
            D = torch.full((M + 2, self.ldd), float("nan"), dtype=self.out, device="cuda")
        layout = {"row": igc.ROW_MAJOR, "col": igc.COL_MAJOR}
        igc.check(GEMM[self.dtype](M, N, K, self.Abuf, self.Abuf.stride(0), layout[self.la], self.Bbuf,
                                   self.Bbuf.stride(0), layout[self.lb], D, self.ldd, igc.out_code(self.out),
                                   epilogue or self.epilogue(), tune, workspace, stream=stream))
        return D

    def check(self, D, what=""):
        M, N, _ = self.dims
        synchronize()
        assert torch.isnan(D[:M, N:].float()).all() and torch.isnan(D[M:].float()).all(), f"{what}: stray store"
        assert_within(D[:M, :N], self.y, self.tol, what)
        if self.pre is not None and not self.backward:
            assert_within(self.pre, self.z, self.ez, what + " pre")
            assert torch.isnan(self.pre_buf[:M, N:].float()).all() and torch.isnan(self.pre_buf[M:].float()).all()


SIZES = [(1, 1, 1), (1, 24, 200), (3, 17, 33), (16, 130, 64), (17, 257, 129), (33, 40, 1000), (64, 300, 260),
         (65, 65, 65), (129, 127, 72), (200, 96, 264), (300, 520, 100)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_sizes_and_layouts(M, N, K, dtype):
    for la, lb in itertools.product(("row", "col"), ("row", "col")):
        say(f"epilogue {M}x{N}x{K} {dtype} {la} {lb}")
        p = Problem(M, N, K, dtype, la=la, lb=lb, act="gelu", bias=dtype, seed=M + N + K)
        p.check(p.run(), f"{M}x{N}x{K} {la} {lb}")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [5, 40, 150])
def test_activations_both_directions(act, M):
    for dtype, out, res, pre in (("bf16", "f32", "f32", "f32"), ("fp16", "fp16", "in", "in"), ("bf16", "bf16", None, "in"),
                                 ("bf16", "f16", "bf16", None)):
        say(f"activation {act} M {M} {dtype} {out}")
        p = Problem(M, 203, 96, dtype, out, act=act, residual=res, pre=pre, seed=M)
        p.check(p.run(), f"{act} forward {dtype} {out}")
        p = Problem(M, 203, 96, dtype, out, act=act, residual=res, pre=pre or "in", backward=True, bias=None, lb="row",
                    seed=M + 1)
        p.check(p.run(), f"{act} backward {dtype} {out}")


@pytest.mark.parametrize("M", [1, 20, 70])
def test_parts_left_out(M):
    """Every combination of bias, residual and pre, and none of them."""
    for bias, res, pre in itertools.product((None, "f32", "f16"), (None, "in", "f32"), (None, "in")):
        say(f"parts M {M} bias {bias} residual {res} pre {pre}")
        p = Problem(M, 72, 40, "fp16", act="silu", bias=bias, residual=res, pre=pre, seed=3)
        p.check(p.run(), f"{bias} {res} {pre}")


def test_empty_sums_and_outputs():
    for M in (2, 100):
        p = Problem(M, 50, 0, act="relu", residual="in", pre="in")
        p.check(p.run(), "K = 0")
    e = igc.Epilogue(act="relu")
    for M, N in ((0, 8), (8, 0)):
        assert igc.gemm_bf16_epilogue(M, N, 8, None, 8, 0, None, 8, 0, None, 8, igc.OUT_F32, e) == igc.IGC_OK


@pytest.mark.parametrize("M,N,K,tune", [
    (1000, 500, 8192, None),                                    # stream-K without an epilogue: a K split here
    (140, 136, 1024, (128, 128, 64, 4, 8, 16, 0, 4, 3)),        # explicit splits, ragged tiles
    (260, 300, 2056, (256, 256, 64, 2, 8, 16, 1, 4, 2)),
    (300, 200, 515, (256, 128, 64, 3, 8, 16, 0, 4, 2)),
])
def test_split_k(M, N, K, tune):
    t = igc.tune(tune[:8], k_splits=tune[8]) if tune else None
    for backward in (False, True):
        say(f"split {M}x{N}x{K} {tune} backward {backward}")
        p = Problem(M, N, K, "bf16", act="gelu_tanh", pre="in", backward=backward, seed=5)
        need = igc.igc_epilogue_workspace_bytes(igc.OP_GEMM, M, N, K, t)
        assert need > 0
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        before = igc.igc_pool_allocations()
        first = p.run(t, ws)
        p.check(first, "split")
        assert igc.igc_pool_allocations() == before
        short = ws[:need - 256]
        with pytest.raises(igc.IgcError):
            p.run(t, short)
        again = p.run(t)  # the pool's workspace: the same bits
        synchronize()
        assert torch.equal(first[:M, :N], again[:M, :N]) and igc.igc_pool_allocations() == before + 1


def test_few_rows_split_along_k():
    for lb, N, K in (("col", 40, 9000), ("row", 300, 12345), ("row", 2050, 4100)):
        for M in (1, 30, 64):
            say(f"few rows split {lb} {M}x{N}x{K}")
            p = Problem(M, N, K, "bf16", lb=lb, act="silu", pre="in", seed=7)
            p.check(p.run(), f"few rows {lb} {M}x{N}x{K}")


def test_tiles_of_every_configuration():
    """Each configuration built with the epilogue, on sizes that leave edge tiles."""
    for cfg in igc.tunes(igc.SCOPE_ALL | igc.SCOPE_EPILOGUE):
        t = igc.tune(cfg)
        for lb, K in (("col", 136), ("row", 129)):
            for backward in (False, True):
                say(f"tile {cfg} {lb} K {K} backward {backward}")
                p = Problem(cfg[0] + 40, cfg[1] + 24, K, "bf16", lb=lb, act="gelu", pre="in", backward=backward, seed=11)
                p.check(p.run(t), f"{cfg} {lb} {backward}")


def test_residual_and_pre_in_place():
    """The residual may be the output, and so may the pre that the backward form reads."""
    for M in (9, 150, 300):
        for tune in (None, igc.tune((128, 128, 64, 4, 8, 16, 0, 4), k_splits=2) if M > 64 else None):
            p = Problem(M, 136, 264, "bf16", act="silu", residual="in", seed=M)
            D = torch.full((M + 2, p.ldd), float("nan"), dtype=torch.bfloat16, device="cuda")
            D[:M, :136] = p.res
            p.check(p.run(tune, D=D, epilogue=p.epilogue(residual=D)), "residual in place")
            p = Problem(M, 136, 264, "bf16", act="silu", residual=None, pre="in", backward=True, seed=M)
            D = torch.full((M + 2, p.ldd), float("nan"), dtype=torch.bfloat16, device="cuda")
            D[:M, :136] = p.pre
            p.pre = D
            p.check(p.run(tune, D=D), "pre in place")


def test_infinities_and_nan_stay_in_their_row_and_column():
    for M in (20, 150):
        p = Problem(M, 100, 72, "bf16", act="relu", residual=None, bias=None, seed=1)
        p.Abuf[3, 5] = float("inf")
        p.Abuf[7, 6] = float("nan")
        p.Bbuf[11, 7] = float("nan")
        D = p.run()
        synchronize()
        y = D[:M, :100]
        keep = torch.ones(M, 100, dtype=torch.bool, device="cuda")
        keep[3], keep[7], keep[:, 11] = False, False, False
        assert_within(y[keep], p.y[keep], p.tol[keep], "rows and columns without a NaN")
        assert torch.isnan(y[7]).all() and torch.isnan(y[:, 11]).all()
        row = torch.cat([y[3, :11], y[3, 12:]])
        assert ((row == 0) | (row == float("inf"))).all()  # relu of -inf and inf
    # the largest finite values do not turn into NaN on the way
    for act in ACTS:
        D = torch.empty(1, 8, dtype=torch.bfloat16, device="cuda")
        bias = torch.tensor([1e30, -1e30, 1e38, -1e38, 3e19, -3e19, 50.0, -50.0], device="cuda")
        A = torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda")
        igc.check(igc.gemm_bf16_epilogue(1, 8, 8, A, 8, 0, A.expand(8, 8).contiguous(), 8, 1, D, 8, igc.OUT_BF16,
                                         igc.Epilogue(act=act, bias=bias)))
        pre = bias.to(torch.bfloat16).reshape(1, 8).contiguous()
        one = torch.ones(1, 8, dtype=torch.bfloat16, device="cuda")
        dz = torch.empty_like(one)
        igc.check(igc.epilogue_backward_bf16(1, 8, act, one, 8, pre, 8, dz, 8, None, 0))
        synchronize()
        assert torch.isfinite(D.float()).all() and torch.isfinite(dz.float()).all(), act
        want = act_grad64(pre.double(), act)
        assert_within(dz, want, torch.full_like(want, GRAD_ABS), act)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_plain_epilogue_equals_the_product(dtype):
    """With nothing in the epilogue, the same bits as the product without one (same tiles, same order)."""
    M, N, K = 300, 520, 320
    p = Problem(M, N, K, dtype, bias=None, residual=None, pad=0)
    t = igc.tune((256, 256, 64, 2, 8, 16, 1, 4))
    D, C = p.run(t), torch.empty(M, p.ldd, dtype=p.out, device="cuda")
    f = igc.gemm_bf16_ex if dtype == "bf16" else igc.gemm_fp16_ex
    igc.check(f(M, N, K, p.Abuf, p.Abuf.stride(0), 0, p.Bbuf, p.Bbuf.stride(0), 1, C, p.ldd, igc.out_code(p.out), t))
    synchronize()
    assert torch.equal(D[:M, :N], C[:, :N])


def test_captured_calls_replay():
    """Few rows, whole tiles and a K split with the caller's workspace, captured and replayed on new inputs with eager
    work in between; two graphs that share one workspace run one after the other."""
    ws = torch.empty(igc.igc_epilogue_workspace_bytes(igc.OP_GEMM, 500, 500, 8192), dtype=torch.uint8, device="cuda")
    problems = [Problem(1, 300, 8192, "bf16", act="silu", seed=21), Problem(500, 500, 8192, "bf16", act="gelu", seed=22),
                Problem(300, 300, 128, "fp16", act="relu", pre="in", seed=23)]
    outs, graphs = [], []
    for p in problems:
        outs.append(p.run(workspace=ws))
        synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.run(workspace=ws, D=outs[-1])
        graphs.append(g)
    for turn in range(3):
        for p, D, g in zip(problems, outs, graphs):
            new = Problem(*p.dims, p.dtype, act=p.act, pre="in" if p.pre is not None else None, seed=100 + turn)
            for name in ("Abuf", "Bbuf", "bias", "res"):
                getattr(p, name).copy_(getattr(new, name))
            p.z, p.ez, p.y, p.tol = new.z, new.ez, new.y, new.tol
            D.fill_(float("nan"))
            g.replay()
            p.check(D, f"replay {turn}")
            eager = p.run(workspace=ws)
            synchronize()
            assert torch.equal(eager[:p.dims[0], :p.dims[1]], D[:p.dims[0], :p.dims[1]])


def test_pool_workspace_is_refused_under_capture():
    p = Problem(500, 500, 8192, "bf16", act="gelu", seed=22)
    p.run()
    synchronize()
    g = torch.cuda.CUDAGraph()
    D = torch.empty(502, p.ldd, dtype=torch.bfloat16, device="cuda")
    with torch.cuda.graph(g):
        with pytest.raises(igc.IgcError) as e:
            p.run(D=D)
        D.zero_()
    assert e.value.status == igc.IGC_ERR_UNSUPPORTED


def test_two_streams_at_once():
    a, b = Problem(1, 500, 8192, "bf16", act="silu", seed=31), Problem(40, 700, 8192, "bf16", lb="row", seed=32)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    da = torch.full((3, a.ldd), float("nan"), dtype=a.out, device="cuda")
    db = torch.full((42, b.ldd), float("nan"), dtype=b.out, device="cuda")
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(D=da, stream=sa)
        b.run(D=db, stream=sb)
    torch.cuda.synchronize()
    a.check(da, "stream a")
    b.check(db, "stream b")


def test_two_threads_at_once():
    """Calls from two host threads, each with its own stream and problem, plain entry points (pool workspaces)."""
    import threading
    problems = [Problem(30, 300, 9000, "bf16", lb="row", act="gelu", seed=41), Problem(400, 300, 8192, "fp16", seed=42)]
    outs = [torch.full((p.dims[0] + 2, p.ldd), float("nan"), dtype=p.out, device="cuda") for p in problems]
    torch.cuda.synchronize()
    failed = []

    def work(p, D, stream):
        try:
            for _ in range(20):
                p.run(D=D, stream=stream)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(p, D, torch.cuda.Stream())) for p, D in zip(problems, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for p, D in zip(problems, outs):
        p.check(D, "threads")


def test_built_in_choices():
    """Sizes that the built-in choice gives to each kind of tile and schedule, ragged."""
    for M, N, K in ((1300, 4104, 72), (4000, 4100, 40), (129, 1025, 2056), (60, 9000, 104), (16, 9001, 72), (64, 6250, 64)):
        for lb in ("col", "row"):
            say(f"built-in {M}x{N}x{K} {lb}")
            p = Problem(M, N, K, "bf16", lb=lb, act="silu", pre="in" if M != 1300 else None, seed=M)
            p.check(p.run(), f"{M}x{N}x{K} {lb}")


def test_parameters_at_odd_addresses():
    """bias needs only its own type's alignment."""
    for M in (3, 100):
        p = Problem(M, 72, 64, "fp16", bias="f16", seed=6)
        shifted = torch.empty(80, dtype=torch.float16, device="cuda")
        shifted[3:75] = p.bias
        p.bias = shifted[3:75]
        p.check(p.run(), "odd bias")


def test_long_leading_dimensions():
    """Rows so far apart that offsets within the output, residual and pre pass 32 bits, and within a tile nearly 31."""
    M, N, K, ld = 600, 64, 64, (1 << 21) - 8
    g = generator(8)
    A, B = normal(g, M, K, dtype=torch.bfloat16).cuda(), normal(g, N, K, scale=0.125, dtype=torch.bfloat16).cuda()
    R = normal(g, M, N, dtype=torch.bfloat16).cuda()
    bufs = [torch.empty(M * ld, dtype=torch.bfloat16, device="cuda") for _ in range(3)]  # 2.5 GB each, hardly touched
    res, pre, D = (b.view(M, ld) for b in bufs)
    res[:, :N] = R
    igc.check(igc.gemm_bf16_epilogue(M, N, K, A, K, 0, B, K, 1, D, ld, igc.OUT_BF16,
                                     igc.Epilogue(act="silu", residual=res, pre=pre)))
    synchronize()
    a, b = A.double(), B.double()
    z, S = a @ b.t(), a.abs() @ b.abs().t()
    ez, y = (K + 2) * U32 * S, act64(z, "silu")
    assert_within(pre[:, :N], z, ez, "pre")
    assert_within(D[:, :N], y + R.double(), ez * ACT_LIP + ACT_REL * (1 + z * z) * y.abs() + U32 * (y.abs() + R.double().abs()))
    far = (1 << 22)  # 256 rows of it pass 2^31 bytes: refused
    tune = igc.tune((256, 256, 64, 2, 8, 16, 1, 4))
    for e in (igc.Epilogue(residual=1 << 20, ldr=far, residual_type=igc.OUT_BF16), igc.Epilogue(pre=1 << 20, ldp=far, pre_type=1)):
        assert igc.gemm_bf16_epilogue_ex(M, N, K, A, K, 0, B, K, 1, D, ld, igc.OUT_BF16, e, tune) == igc.IGC_ERR_UNSUPPORTED


def test_long_weights_of_few_rows():
    """Weights of more than 2^32 bytes in both layouts; the last rows and columns are checked."""
    M, N, K = 2, 70000, 32768
    A = normal(generator(1), M, K, dtype=torch.bfloat16).cuda()
    for lb in ("col", "row"):
        say(f"long weights {lb}")
        B = torch.empty((N, K) if lb == "col" else (K, N), dtype=torch.bfloat16, device="cuda")
        B.normal_(generator=torch.Generator(device="cuda").manual_seed(3))
        D = torch.full((M, N), float("nan"), device="cuda")
        igc.check(igc.gemm_bf16_epilogue(M, N, K, A, K, 0, B, B.stride(0), 1 if lb == "col" else 0, D, N, igc.OUT_F32,
                                         igc.Epilogue(act="none")))
        synchronize()
        assert torch.isfinite(D).all()
        for n0 in (0, 34990, N - 24):
            b = (B[n0:n0 + 24] if lb == "col" else B[:, n0:n0 + 24].t()).double()
            a = A.double()
            assert_within(D[:, n0:n0 + 24].contiguous(), a @ b.t(), (K + 2) * U32 * (a.abs() @ b.abs().t()), f"{lb} {n0}")
        del B


# ---- convolution ------------------------------------------------------------------------------------------------------

CONV = {"bf16": igc.conv2d_nhwc_implicit_gemm_epilogue_ex, "fp16": igc.conv2d_nhwc_implicit_gemm_epilogue_fp16_ex}


def conv_case(N, H, W, C, K, R, S, stride, pad, dtype, act, out=None, bias="f32", residual=True, pre=True, tune=None,
              seed=0):
    g, t = generator(seed), DT[dtype]
    P, Q = igc.conv_out_hw(H, W, R, S, stride, stride, pad, pad)
    x, w = normal(g, N, H, W, C, dtype=t).cuda(), normal(g, K, R, S, C, scale=(R * S * C) ** -0.5, dtype=t).cuda()
    b = normal(g, K, scale=0.5, dtype=DT[bias]).cuda() if bias else None
    res = normal(g, N, P, Q, K, dtype=t).cuda() if residual else None
    out_t = DT[out or dtype]
    y = torch.full((N * P * Q + 1, K), float("nan"), dtype=out_t, device="cuda")
    z16 = torch.full((N * P * Q + 1, K), float("nan"), dtype=t, device="cuda") if pre else None
    igc.check(CONV[dtype](N, H, W, C, K, R, S, stride, stride, pad, pad, 1, 1, x, w, y, igc.out_code(out_t),
                          igc.Epilogue(act=act, bias=b, residual=res, pre=z16), tune))
    synchronize()
    xd, wd = x.double().permute(0, 3, 1, 2), w.double().permute(0, 3, 1, 2).reshape(K, -1)
    cols = torch.nn.functional.unfold(xd, (R, S), padding=pad, stride=stride).transpose(1, 2).reshape(N * P * Q, -1)
    z, Sabs = cols @ wd.t(), cols.abs() @ wd.abs().t()
    if bias:
        z, Sabs = z + b.double(), Sabs + b.double().abs()
    ez = (R * S * C + 2) * U32 * Sabs
    want = act64(z, act)
    tol = ez * ACT_LIP + ACT_REL * (1 + z * z) * want.abs()
    if residual:
        r = res.double().reshape(-1, K)
        tol, want = tol + U32 * (want.abs() + r.abs()), want + r
    assert_within(y[:-1], want, tol, "y")
    assert torch.isnan(y[-1].float()).all(), "store past the last pixel"
    if pre:
        assert_within(z16[:-1], z, ez, "pre")
        assert torch.isnan(z16[-1].float()).all()


@pytest.mark.parametrize("geometry", [
    (2, 9, 7, 32, 24, 3, 3, 1, 1), (1, 5, 5, 8, 8, 1, 1, 1, 0), (3, 14, 13, 64, 64, 3, 3, 2, 1),
    (2, 12, 12, 128, 13, 3, 3, 1, 1),     # filters not a multiple of 8: rows of y no vector fits
    (2, 10, 11, 72, 300, 3, 3, 1, 1), (1, 20, 20, 16, 40, 17, 1, 1, 0),  # a filter taller than 16 taps
])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_convolution(geometry, dtype):
    for act, out, bias, res, pre in (("silu", None, "f32", True, True), ("relu", "f32", dtype, False, False),
                                     ("none", None, None, True, False)):
        say(f"conv {geometry} {dtype} {act}")
        conv_case(*geometry, dtype, act, out, bias, res, pre, seed=sum(geometry))


def test_convolution_tiles():
    for cfg in igc.tunes(igc.SCOPE_EPILOGUE):
        for geometry in ((2, 17, 16, 64, 264, 3, 3, 1, 1), (2, 17, 16, 72, 72, 3, 3, 1, 1), (1, 30, 24, 8, 40, 18, 2, 1, 0)):
            say(f"conv tile {cfg} {geometry}")
            conv_case(*geometry, "bf16", "gelu_tanh", tune=igc.tune(cfg), seed=2)
            conv_case(*geometry, "fp16", "gelu", tune=igc.tune(cfg, k_splits=2) if cfg[:2] == (128, 128) else None, seed=3)


# ---- the epilogue's gradient --------------------------------------------------------------------------------------


def back_case(M, N, dtype, act, dz=True, dbias="f32", pad=8, seed=0, workspace=None):
    g, t = generator(seed), DT[dtype]
    ld = round8(N) + pad
    d, _ = padded(normal(g, M, N, dtype=t), ld)
    pre, _ = padded(normal(g, M, N, scale=2.0, dtype=t), ld)
    out = torch.full((M + 2, ld), float("nan"), dtype=t, device="cuda") if dz else None
    db = torch.full((N,), float("nan"), dtype=DT[dbias], device="cuda") if dbias else None
    igc.check(BACK[dtype](M, N, act, d, ld, pre if act != "none" else None, ld, out, ld, db,
                          igc.out_code(DT[dbias or "f32"]), workspace=workspace))
    synchronize()
    grad = act_grad64(pre.double(), act)
    want = d.double() * grad
    tol = d.double().abs() * (GRAD_ABS if act not in ("none", "relu") else 0.0) + U32 * want.abs()
    if dz:
        assert_within(out[:M, :N], want, tol, f"dz {act}")
        assert torch.isnan(out[:M, N:].float()).all() and torch.isnan(out[M:].float()).all()
    if dbias:
        assert_within(db, want.sum(0), tol.sum(0) + M * U32 * want.abs().sum(0), f"dbias {act}")
    return db


@pytest.mark.parametrize("M,N", [(1, 1), (1, 1000), (3, 8), (100, 7), (257, 33), (1000, 130), (2049, 256), (5000, 520)])
def test_epilogue_backward(M, N):
    for act in ACTS:
        for dtype, dz, db in (("bf16", True, "f32"), ("fp16", True, "fp16"), ("bf16", False, "bf16"), ("fp16", True, None)):
            say(f"epilogue_backward {M}x{N} {act} {dtype} {dz} {db}")
            back_case(M, N, dtype, act, dz, db, seed=M)


def test_epilogue_backward_workspace_and_empty():
    M, N = 4000, 300
    need = igc.igc_epilogue_backward_workspace_bytes(M, N)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    before = igc.igc_pool_allocations()
    a = back_case(M, N, "bf16", "gelu", workspace=ws)
    assert igc.igc_pool_allocations() == before
    assert torch.equal(a, back_case(M, N, "bf16", "gelu"))  # the same bits with the pool's
    db = torch.full((24,), float("nan"), device="cuda")
    igc.check(igc.epilogue_backward_bf16(0, 24, "silu", None, 24, None, 24, None, 24, db, igc.OUT_F32))
    synchronize()
    assert (db == 0).all()


def test_epilogue_backward_in_place():
    M, N = 333, 72
    g = generator(4)
    d, pre = normal(g, M, N, dtype=torch.bfloat16).cuda(), normal(g, M, N, dtype=torch.bfloat16).cuda()
    want = d.double() * act_grad64(pre.double(), "silu")
    tol = d.double().abs() * GRAD_ABS + U32 * want.abs()
    for target in ("d", "pre"):
        x, p = d.clone(), pre.clone()
        o = x if target == "d" else p
        igc.check(igc.epilogue_backward_bf16(M, N, "silu", x, N, p, N, o, N, None, 0))
        synchronize()
        assert_within(o, want, tol, target)


def test_linear_layer_gradients_against_differences():
    """loss = sum(dy * D) of one layer: the library's gradients along random directions against central differences of
    the definition in 64 bits.  The gradient is linear in dz, which is rounded once to 16 bits, as pre is."""
    M, N, K, act, t = 70, 48, 40, "gelu", torch.float16
    g = generator(9)
    x, w = normal(g, M, K, dtype=t).cuda(), normal(g, N, K, scale=K ** -0.5, dtype=t).cuda()
    b, dy = normal(g, N, scale=0.5, dtype=t).cuda(), normal(g, M, N, dtype=t).cuda()
    y, pre, dz = (torch.empty(M, N, dtype=t, device="cuda") for _ in range(3))
    db = torch.empty(N, device="cuda")
    dx, dw = torch.empty(M, K, device="cuda"), torch.empty(N, K, device="cuda")
    igc.check(igc.gemm_fp16_epilogue(M, N, K, x, K, 0, w, K, 1, y, N, igc.OUT_F16,
                                     igc.Epilogue(act=act, bias=b, pre=pre)))
    igc.check(igc.epilogue_backward_fp16(M, N, act, dy, N, pre, N, dz, N, db, igc.OUT_F32))
    igc.check(igc.gemm_fp16(M, K, N, dz, N, 0, w, K, 0, dx, K, igc.OUT_F32))
    igc.check(igc.gemm_fp16(N, K, M, dz, N, 1, x, K, 0, dw, K, igc.OUT_F32))
    synchronize()
    xd, wd, bd, gd = x.double(), w.double(), b.double(), dy.double()

    def loss(a, c, e):
        return (gd * act64(a @ c.t() + e, act)).sum()

    z = xd @ wd.t() + bd
    zrow = half_step(z, t) + (K + 2) * U32 * (xd.abs() @ wd.abs().t() + bd.abs())  # what pre is off by
    true = gd * act_grad64(z, act)
    edz = gd.abs() * (ACT_CURVE * zrow + GRAD_ABS) + half_step(true, t) * 1.01
    etol = {"x": edz @ wd.abs() + N * U32 * (true.abs() @ wd.abs()),
            "w": edz.t() @ xd.abs() + M * U32 * (true.abs().t() @ xd.abs()),
            "b": gd.abs().mul(ACT_CURVE * zrow + GRAD_ABS).sum(0) + M * U32 * true.abs().sum(0)}
    h = 1e-5
    for name, grad in (("x", dx), ("w", dw), ("b", db)):
        v = torch.randn(grad.shape, generator=generator(1), dtype=torch.float64).cuda()
        at = {"x": xd, "w": wd, "b": bd}
        up, down = dict(at), dict(at)
        up[name], down[name] = at[name] + h * v, at[name] - h * v
        diff = (loss(*up.values()) - loss(*down.values())) / (2 * h)
        got, tol = (grad.double() * v).sum(), (etol[name] * v.abs()).sum() + 1e-6 * diff.abs() + 1e-6
        assert (got - diff).abs() <= tol, (name, float(got), float(diff), float(tol))


# ---- schedules in parts ---------------------------------------------------------------------------------------------

GEMM_TILES = [c for c in igc.tunes(igc.SCOPE_EPILOGUE) if c in igc.tunes(igc.SCOPE_ALL)]


@pytest.mark.parametrize("cfg", GEMM_TILES, ids=str)
def test_parts_of_every_tile(cfg):
    """K splits of each configuration: every operand layout, edge tiles, rows no vector fits, K not a multiple of 8."""
    for M, N, K, la, lb, dtype in ((261, 133, 1030, "row", "col", "bf16"), (70, 300, 777, "row", "row", "fp16"),
                                   (130, 68, 641, "col", "col", "bf16"), (200, 259, 1024, "col", "row", "fp16")):
        for s in (2, 3):
            say(f"parts {cfg} {M}x{N}x{K} {la} {lb} {dtype} {s}")
            p = Problem(M, N, K, dtype, la=la, lb=lb, act="gelu_tanh", pre="out", seed=M + s)
            p.check(p.run(tune=igc.tune(cfg, k_splits=s)), f"{cfg} {M}x{N}x{K} in {s}")


@pytest.mark.parametrize("cfg", GEMM_TILES, ids=str)
def test_k_tails_of_every_tile(cfg):
    """The last K % 8, with NaN behind every row: K below 8, around a K tile, and parts that are a tail alone."""
    for K in (1, 5, 7, 9, 63, 65, 517, 1030):
        for la, lb in itertools.product(("row", "col"), repeat=2):
            say(f"tail {cfg} {K} {la} {lb}")
            p = Problem(133, 75, K, "bf16" if K % 2 else "fp16", la=la, lb=lb, act="silu", pre="in", seed=K)
            p.check(p.run(tune=igc.tune(cfg)), f"{cfg} {K} {la} {lb}")
            if K > 500:
                for s in (2, 3, 5):
                    p.check(p.run(tune=igc.tune(cfg, k_splits=s)), f"{cfg} {K} {la} {lb} in {s}")
        q = Problem(70, 130, K, "fp16", lb="row", act="gelu", backward=True, seed=K)
        q.check(q.run(tune=igc.tune(cfg)), f"{cfg} {K} backward")


@pytest.mark.parametrize("cfg", igc.tunes(igc.SCOPE_EPILOGUE), ids=str)
def test_convolution_parts_of_every_tile(cfg):
    """The same of the convolution, with filter counts that no vector fits."""
    for geometry in ((2, 12, 12, 128, 13, 3, 3, 1, 1), (1, 17, 16, 72, 300, 3, 3, 1, 1), (2, 11, 9, 256, 72, 1, 1, 1, 0)):
        for s in (1, 2, 3):
            say(f"conv parts {cfg} {geometry} {s}")
            conv_case(*geometry, "bf16", "silu", tune=igc.tune(cfg, k_splits=s if s > 1 else 0), seed=s)
            conv_case(*geometry, "fp16", "relu", residual=False, tune=igc.tune(cfg, k_splits=s if s > 1 else 0), seed=s)


def test_built_in_choices_of_small_outputs():
    """Sizes that take 64-row tiles, whole and in parts, and the convolution's 64-column tiles."""
    for M, N, K in ((200, 300, 100), (1000, 1500, 72), (65, 1, 8), (300, 300, 3001), (77, 6230, 3061), (1990, 1020, 136)):
        for la, lb in (("row", "col"), ("row", "row"), ("col", "row"), ("col", "col")):
            say(f"built-in {M}x{N}x{K} {la} {lb}")
            p = Problem(M, N, K, "fp16", la=la, lb=lb, act="gelu", pre="in" if K == 100 else None, seed=K)
            p.check(p.run(), f"{M}x{N}x{K} {la} {lb}")
    for geometry in ((2, 30, 20, 48, 72, 3, 3, 1, 1), (1, 14, 14, 256, 264, 3, 3, 1, 1), (9, 57, 33, 40, 296, 1, 1, 1, 0),
                     (3, 9, 9, 8, 5, 1, 1, 1, 0)):
        say(f"built-in conv {geometry}")
        conv_case(*geometry, "bf16", "gelu_tanh", seed=4)


def test_few_rows_and_tiles_meet():
    """Row counts, widths and depths on both sides of where the kernel of few rows gives way to tiles."""
    for M in (1, 8, 9, 16, 17, 20, 21, 32, 33):
        for N, K in ((40, 2048), (40, 2056), (8200, 24), (16400, 16), (33000, 8), (24, 6200)):
            for lb in ("col", "row"):
                say(f"few rows {M}x{N}x{K} {lb}")
                p = Problem(M, N, K, "bf16", lb=lb, act="silu", pre="in" if M in (9, 20) else None, seed=M)
                p.check(p.run(), f"{M}x{N}x{K} {lb}")


# ---- extreme values -------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("act", ACTS)
def test_activation_over_the_whole_range(act):
    """An empty sum leaves z = bias: every binade of fp32, both signs, and the neighbourhood of 0.

    Forward, |error| <= ACT_REL * (1 + z^2) * |act(z)| where the exponential's rounding counts (|z| < 15; beyond it a
    tail is below 2^-126 or the result is z to the last bit), plus |z| * 2^-125 for tails below the normal numbers, which
    the hardware's exp2 and reciprocal flush.  Backward, GRAD_ABS and the same flushed tails (|z| * 2^-125 < 2^-120)."""
    z = torch.cat([torch.ldexp(torch.linspace(1, 2, 9)[:-1].double(), torch.arange(-126, 127).double()[:, None]).reshape(-1),
                   torch.linspace(0, 15, 4001).double()]).float()
    z = torch.cat([z, -z, torch.tensor([float("nan"), float("inf")])]).contiguous()
    N = z.numel()
    zd = z.double()
    A = torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda")
    D = torch.full((2, (N + 7) // 8 * 8), 7.0, device="cuda")
    b = z.cuda()
    igc.check(igc.gemm_bf16_epilogue(1, N, 0, A, 8, 0, A, D.stride(0), 0, D, D.stride(0), igc.OUT_F32,
                                     igc.Epilogue(act=act, bias=b)))
    synchronize()
    got, want = D[0, :N].double().cpu(), act64(zd, act)
    fin = torch.isfinite(zd) & torch.isfinite(want)
    tol = ACT_REL * (1 + torch.clamp(zd.abs(), max=15) ** 2) * want.abs() + zd.abs() * 2.0 ** -125 + 2.0 ** -125
    assert ((got - want).abs()[fin] <= (tol + U32 * want.abs())[fin]).all()
    assert torch.isnan(got[-2]) and got[-1] == float("inf")
    assert (D[0, N:] == 7.0).all() and (D[1] == 7.0).all()
    pre = torch.zeros(1, D.stride(0), device="cuda")
    pre[0, :N] = b
    D.fill_(7.0)
    ones = torch.ones(N, device="cuda")
    igc.check(igc.gemm_bf16_epilogue(1, N, 0, A, 8, 0, A, D.stride(0), 0, D, D.stride(0), igc.OUT_F32,
                                     igc.Epilogue(act=act, bias=ones, pre=pre, backward=True)))
    synchronize()
    got, want = D[0, :N].double().cpu(), act_grad64(torch.clamp(zd, -1e4, 1e4), act)
    fin = torch.isfinite(zd)
    assert ((got - want).abs()[fin] <= GRAD_ABS).all()
    assert act == "none" or torch.isnan(got[-2])


def test_pinned_tensors_are_read_and_written():
    """Pinned memory is the GPU's to reach: operands, bias, residual and output there give the same bits."""
    for M in (3, 100):
        p = Problem(M, 72, 64, "bf16", act="silu", seed=M)
        want = p.run()
        synchronize()
        pinned = {n: torch.empty(v.shape, dtype=v.dtype, pin_memory=True).copy_(v)
                  for n, v in (("Abuf", p.Abuf), ("Bbuf", p.Bbuf), ("bias", p.bias), ("D", want))}
        res = torch.zeros(M, p.ldd, dtype=p.res.dtype, pin_memory=True)
        res[:, :72].copy_(p.res)
        p.Abuf, p.Bbuf, p.bias, D = (pinned[n] for n in ("Abuf", "Bbuf", "bias", "D"))
        D.fill_(float("nan"))
        p.run(D=D, epilogue=p.epilogue(residual=res))
        synchronize()
        assert torch.equal(D[:M, :72], want[:M, :72].cpu()) and torch.isnan(D[M:].float()).all()


def test_epilogue_backward_of_one_very_long_row():
    """A row so long that a workgroup of 64 columns and 1024 threads for every piece of it would pass 2^32 threads."""
    N = (1 << 28) + 24
    d = torch.empty(1, N, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    db = torch.full((N,), float("nan"), device="cuda")
    say("one long row")
    igc.check(igc.epilogue_backward_bf16(1, N, "silu", d, N, d, N, None, 0, db, igc.OUT_F32))
    synchronize()
    for n0 in range(0, N, 1 << 25):
        v = d[0, n0:n0 + (1 << 25)].double()
        want = v * act_grad64(v, "silu")
        assert_within(db[n0:n0 + (1 << 25)], want, v.abs() * GRAD_ABS + U32 * want.abs(), f"columns from {n0}")


FEW = [  # M, N, K, layout of B, columns of a workgroup: several turns of K a wave and a partial last one
    (1, 16411, 1100, "row", 64), (8, 16400, 2085, "row", 64), (8, 32650, 1100, "row", 128), (3, 33003, 2085, "row", 128),
    (1, 500, 2047, "row", 32), (20, 300, 2045, "row", 32), (7, 700, 1100, "col", 16), (32, 203, 2041, "col", 16),
    (8, 5000, 4099, "col", 16),
]


@pytest.mark.parametrize("M,N,K,lb,cols", FEW)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_kernel_of_few_rows(M, N, K, lb, cols, dtype):
    """Each operand width of the kernel of few rows, which the query says it runs on, over a K of several turns."""
    t = igc.igc_epilogue_default_tune(M, N, K, lb=igc.COL_MAJOR if lb == "col" else igc.ROW_MAJOR)
    assert (t.bm, t.bn, t.k_splits) == (0, cols, 1)
    for backward in (False, True):
        say(f"few rows {M}x{N}x{K} {lb} {dtype} backward {backward}")
        p = Problem(M, N, K, dtype, lb=lb, act="silu" if backward else "gelu", bias="f32", residual="in", pre="in",
                    backward=backward, seed=M + K)
        p.check(p.run(), f"{M}x{N}x{K} {lb} {backward}")


@pytest.mark.parametrize("M,N,K", [(1, 40, 9000), (5, 300, 12345), (8, 1000, 6200), (3, 24, 65531)])
def test_few_rows_in_parts(M, N, K):
    """Parts along K of the kernel of few rows: column-major weights, at most eight rows and a K of 6144 or more."""
    assert igc.igc_epilogue_default_tune(M, N, K).bm == 0 and igc.igc_epilogue_default_tune(M, N, K).k_splits > 1
    for dtype, backward in (("bf16", False), ("fp16", True), ("fp16", False)):
        say(f"few rows in parts {M}x{N}x{K} {dtype} backward {backward}")
        p = Problem(M, N, K, dtype, act="gelu_tanh", pre="in", backward=backward, seed=K)
        ws = torch.empty(igc.igc_epilogue_workspace_bytes(igc.OP_GEMM, M, N, K), dtype=torch.uint8, device="cuda")
        before = igc.igc_pool_allocations()
        D = p.run(workspace=ws)
        p.check(D, f"{M}x{N}x{K} {dtype}")
        assert igc.igc_pool_allocations() == before
        own = p.run()
        synchronize()
        assert torch.equal(own[:M, :N], D[:M, :N]) and igc.igc_pool_allocations() == before + 1
        E = torch.full_like(D, float("nan"))
        E[:M, :N] = p.res
        p.check(p.run(D=E, workspace=ws, epilogue=p.epilogue(residual=E)), "residual in place")
