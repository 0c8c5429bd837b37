"""Group norm with an activation, forward and backward, through the C ABI against its definition in 64 bits: group
widths that no vector fits, one pixel to large images, channel slices, extreme means and values, in-place calls,
caller workspaces, graphs, and the gradient against differences.  Then a residual block made of the library's calls."""
import pytest
import torch

import implicit_gemm_conv_amd as igc
from fused_util import (ACT_CURVE, ACT_LIP, ACT_REL, ACTS, DT, GRAD_ABS, U32, act64, act_grad64, assert_within,
                        generator, half_step, normal)
from gpu_util import say, synchronize

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    igc.lib()


FWD = {"bf16": igc.group_norm_nhwc_bf16_ex, "fp16": igc.group_norm_nhwc_fp16_ex}
BWD = {"bf16": igc.group_norm_nhwc_backward_bf16_ex, "fp16": igc.group_norm_nhwc_backward_fp16_ex}
EPS = 1e-5
# A fp32 sum over a group: every partial is a sum of at most a few hundred terms and the partials are joined the same
# way, so sums are good to 512 * 2^-24 of the sum of their terms' sizes.
SUM = 512 * U32


class Norm:
    """Inputs on the GPU -- x, y, dy, dx being channel slices of wider tensors whose other channels are NaN -- and the
    expected results with their tolerances."""

    def __init__(self, N, H, W, C, G, dtype="bf16", params="f32", act="silu", affine=True, wide=8, seed=0, x=None, eps=EPS):
        g, t = generator(seed), DT[dtype]
        self.dims, self.dtype, self.act, self.ld, self.eps = (N, H, W, C, G), dtype, act, C + wide, eps
        self.params, self.t = DT[params], t
        if x is None:
            x = normal(g, N, H, W, C) * (0.5 + normal(g, C).abs()) + normal(g, C)
        self.x = self.wide(x.to(t))
        self.dy = self.wide(normal(g, N, H, W, C, dtype=t))
        self.gamma = (1 + normal(g, C, scale=0.3)).to(self.params).cuda() if affine else None
        self.beta = normal(g, C, scale=0.3, dtype=self.params).cuda() if affine else None
        xd = self.x[..., :C].double().reshape(N, H * W, G, C // G)
        self.mu = xd.mean((1, 3), keepdim=True) if N else xd.new_zeros(0, 1, G, 1)
        d = xd - self.mu
        var = (d * d).mean((1, 3), keepdim=True)
        self.rs = 1 / torch.sqrt(var + eps)
        self.xh = d * self.rs
        one = torch.ones(C, dtype=torch.float64, device="cuda")
        self.ga = (self.gamma.double() if affine else one).reshape(G, C // G)
        self.be = (self.beta.double() if affine else 0 * one).reshape(G, C // G)
        self.z = self.xh * self.ga + self.be
        # mean: off by SUM of the mean distance from the shift points (about the group's spread) and its own rounding;
        # rstd: SUM of itself; xh then by SUM (1 + |xh|) and the rounding of x - mu next to a large mean
        self.emu = SUM * (d.abs().mean((1, 3), keepdim=True) * 4 + 1e-30) + 4 * U32 * self.mu.abs()
        self.exh = 2 * SUM * (1 + self.xh.abs()) + 8 * U32 * self.mu.abs() * self.rs
        self.ez = self.exh * self.ga.abs() + 3 * U32 * (self.z.abs() + self.be.abs())
        want = act64(self.z, act)
        self.y, self.ey = want, self.ez * ACT_LIP + ACT_REL * (1 + self.z * self.z) * want.abs()

    def wide(self, v):
        N, H, W, C, _ = self.dims
        out = torch.full((N, H, W, self.ld), float("nan"), dtype=v.dtype)
        out[..., :C] = v
        return out.cuda()

    def blank(self):
        N, H, W, C, _ = self.dims
        return torch.full((N, H, W, self.ld), float("nan"), dtype=self.t, device="cuda")

    def inside(self, wide, what):
        N, H, W, C, G = self.dims
        assert torch.isnan(wide[..., C:].float()).all(), f"{what}: stray store"
        return wide[..., :C].reshape(N, H * W, G, C // G)

    def forward(self, y=None, stats=True, workspace=None, x=None, stream=None):
        N, H, W, C, G = self.dims
        y = self.blank() if y is None else y
        mean, rstd = (torch.full((N, G), float("nan"), device="cuda") for _ in range(2)) if stats else (None, None)
        igc.check(FWD[self.dtype](N, H, W, C, G, self.x if x is None else x, self.ld, self.gamma, self.beta,
                                  igc.out_code(self.params), self.eps, self.act, y, self.ld, mean, rstd, workspace,
                                  stream=stream))
        return y, mean, rstd

    def check_forward(self, y, mean, rstd, what=""):
        synchronize()
        assert_within(self.inside(y, what), self.y, self.ey, what + " y")
        if mean is not None:
            assert_within(mean, self.mu[:, 0, :, 0], self.emu[:, 0, :, 0], what + " mean")
            assert_within(rstd, self.rs[:, 0, :, 0], 2 * SUM * self.rs[:, 0, :, 0], what + " rstd")

    def backward(self, dx=None, dy=None, mean=None, rstd=None, workspace=None, grads=True):
        N, H, W, C, G = self.dims
        dx = self.blank() if dx is None else dx
        mean = self.mu[:, 0, :, 0].float().contiguous() if mean is None else mean
        rstd = self.rs[:, 0, :, 0].float().contiguous() if rstd is None else rstd
        dg, db = (torch.full((C,), float("nan"), dtype=self.params, device="cuda") if grads else None for _ in range(2))
        igc.check(BWD[self.dtype](N, H, W, C, G, self.x, self.ld, self.gamma, self.beta, igc.out_code(self.params), mean,
                                  rstd, self.act, self.dy if dy is None else dy, self.ld, dx, self.ld, dg, db, workspace))
        return dx, dg, db

    def expect_backward(self):
        N, H, W, C, G = self.dims
        dy = self.dy[..., :C].double().reshape(self.z.shape)
        dz = dy * act_grad64(self.z, self.act)
        smooth = self.act not in ("none", "relu")
        edz = dy.abs() * (ACT_CURVE * self.ez + GRAD_ABS if smooth else 0.0) + 2 * U32 * dz.abs()
        if self.act == "relu":  # its derivative jumps: a z that rounding may carry over zero may have either
            edz = edz + dy.abs() * (self.z.abs() <= self.ez)
        q, eq = dz * self.ga, edz * self.ga.abs() + 2 * U32 * (dz * self.ga).abs()
        mean = lambda v: v.mean((1, 3), keepdim=True)  # noqa: E731
        c1, c2 = mean(q), mean(q * self.xh)
        ec1 = mean(eq) + SUM * mean(q.abs())
        ec2 = mean(eq * self.xh.abs() + q.abs() * self.exh) + SUM * mean((q * self.xh).abs())
        inner = q - c1 - self.xh * c2
        einner = eq + ec1 + self.xh.abs() * ec2 + self.exh * c2.abs() + 4 * U32 * (q.abs() + c1.abs() + (self.xh * c2).abs())
        dx = self.rs * inner
        edx = self.rs * einner + 4 * U32 * dx.abs()
        chan = lambda v: v.sum((0, 1)).reshape(C)  # noqa: E731
        dg, db = chan(dz * self.xh), chan(dz)
        edg = chan(edz * self.xh.abs() + dz.abs() * self.exh) + 4 * SUM * chan((dz * self.xh).abs())
        edb = chan(edz) + 4 * SUM * chan(dz.abs())
        return (dx, edx), (dg, edg), (db, edb)

    def check_backward(self, dx, dg, db, what=""):
        synchronize()
        (wdx, edx), (wdg, edg), (wdb, edb) = self.expect_backward()
        assert_within(self.inside(dx, what), wdx, edx, what + " dx")
        if dg is not None:
            assert_within(dg, wdg, edg, what + " dgamma")
            assert_within(db, wdb, edb, what + " dbeta")


SHAPES = [
    (1, 1, 1, 8, 1), (1, 1, 1, 8, 8), (2, 1, 3, 16, 4), (3, 5, 7, 40, 4),      # groups of 8, 1, 4 and 10 channels
    (2, 4, 4, 24, 8), (1, 9, 11, 56, 8),                                      # 3 and 7
    (2, 8, 8, 1280, 32), (16, 3, 3, 320, 32), (1, 13, 17, 2056, 1),           # one group over more than one workgroup
    (2, 33, 31, 64, 8), (1, 100, 90, 32, 32), (1, 300, 211, 8, 2), (5, 56, 56, 256, 32), (1, 64, 64, 4096, 64),
    (2, 47, 53, 320, 32), (2, 70, 70, 96, 4), (1, 120, 130, 128, 1),
    (40, 30, 34, 64, 8), (33, 61, 40, 48, 16), (16, 32, 32, 640, 32), (9, 128, 120, 64, 64), (130, 40, 33, 40, 4),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_forward_and_backward(shape, dtype):
    for k, act in enumerate(("none", "silu") if shape[0] * shape[1] * shape[2] > 2000 else ACTS):
        for params in ("f32", dtype):
            say(f"group norm {shape} {dtype} {act} {params}")
            p = Norm(*shape, dtype=dtype, params=params, act=act, seed=k + sum(shape))
            p.check_forward(*p.forward(), f"{shape} {act}")
            p.check_backward(*p.backward(), f"{shape} {act}")


def test_without_parameters_statistics_or_parameter_gradients():
    for shape in ((2, 6, 6, 48, 6), (2, 60, 60, 48, 6)):
        p = Norm(*shape, affine=False, act="gelu")
        p.check_forward(*p.forward(stats=False))
        p.check_backward(*p.backward(grads=False))
        q = Norm(*shape, affine=False, act="gelu")
        p.check_forward(*q.forward())


def test_no_images():
    p = Norm(0, 4, 4, 16, 2)
    p.forward()
    _, dg, db = p.backward()
    synchronize()
    assert (dg == 0).all() and (db == 0).all()


def test_large_means_constants_and_outliers():
    for shape in ((2, 8, 8, 64, 8), (2, 64, 64, 64, 8)):
        N, H, W, C, G = shape
        g = generator(5)
        base = normal(g, N, H, W, C)
        say(f"means {shape}")
        for x in (base + 200, base * 0.01 - 3, base + 30 * torch.arange(C)):
            p = Norm(*shape, x=x, dtype="fp16", act="none")
            p.check_forward(*p.forward(), "large mean")
            p.check_backward(*p.backward(), "large mean")
        x = base.clone()
        x[:, 0, 0, :] = 3000.0  # the first value of every channel, which shifts its sums
        x[0, 3, 5, 7] = -20000.0
        p = Norm(*shape, x=x, dtype="fp16", act="none")
        p.check_forward(*p.forward(), "outliers")
        # a constant image: variance 0 exactly
        p = Norm(*shape, x=torch.full((N, H, W, C), 1.5), act="none")
        y, mean, rstd = p.forward()
        p.check_forward(y, mean, rstd, "constant")
        assert (mean == 1.5).all()
        assert_within(rstd, torch.full_like(rstd, EPS ** -0.5).double(), 4 * U32 * torch.full_like(rstd, EPS ** -0.5).double())


def test_nan_and_infinity_stay_in_their_group():
    for shape in ((2, 8, 8, 64, 8), (2, 64, 64, 64, 8), (2, 20, 20, 40, 4)):
        N, H, W, C, G = shape
        p = Norm(*shape, act="silu")
        x = p.x.clone()
        x[0, 1, 2, 0] = float("nan")
        x[1, 0, 0, C - 1] = float("inf")
        y, mean, rstd = p.forward(x=x)
        synchronize()
        v = p.inside(y, "nan")
        assert torch.isnan(v[0, :, 0].float()).all() and torch.isnan(v[1, :, G - 1].float()).all()
        keep = torch.ones(N, G, dtype=torch.bool, device="cuda")
        keep[0, 0], keep[1, G - 1] = False, False
        sel = keep[:, None, :, None].expand(v.shape)
        assert_within(v[sel], p.y[sel], p.ey[sel], "other groups")


def test_in_place():
    for shape in ((2, 8, 8, 64, 8), (3, 70, 64, 64, 8), (2, 9, 9, 40, 4)):
        p = Norm(*shape, act="gelu")
        y, mean, rstd = p.forward(y=(x := p.x.clone()), x=x)
        p.check_forward(y, mean, rstd, "y = x")
        d = p.dy.clone()
        p.check_backward(*p.backward(dx=d, dy=d), "dx = dy")
        keep = p.x
        p.x = keep.clone()
        out = p.backward(dx=p.x)
        p.check_backward(*out, "dx = x")


def test_pixels_far_apart():
    """A channel slice of a tensor so wide that offsets pass 32 bits, in one workgroup a slab and in chunks."""
    for (N, H, W, C, G), ld in (((2, 64, 64, 32, 4), 300000), ((2, 40, 40, 64, 2), 700000)):
        g = generator(3)
        x = normal(g, N, H, W, C, dtype=torch.bfloat16).cuda()
        wide = torch.empty(N * H * W * ld, dtype=torch.bfloat16, device="cuda").view(N, H, W, ld)  # hardly touched
        wide[..., :C] = x
        gamma = torch.ones(C, device="cuda")
        y, z, dx, dz = (torch.empty_like(x) for _ in range(4))
        mean, rstd = (torch.empty(N, G, device="cuda") for _ in range(2))
        igc.check(igc.group_norm_nhwc_bf16(N, H, W, C, G, x, C, gamma, None, 0, EPS, "silu", y, C, mean, rstd))
        igc.check(igc.group_norm_nhwc_bf16(N, H, W, C, G, wide, ld, gamma, None, 0, EPS, "silu", z, C))
        igc.check(igc.group_norm_nhwc_backward_bf16(N, H, W, C, G, x, C, gamma, None, 0, mean, rstd, "silu", y, C, dx, C))
        igc.check(igc.group_norm_nhwc_backward_bf16(N, H, W, C, G, wide, ld, gamma, None, 0, mean, rstd, "silu", y, C, dz, C))
        synchronize()
        assert torch.equal(y, z) and torch.equal(dx, dz)
        igc.check(igc.group_norm_nhwc_bf16(N, H, W, C, G, wide, ld, gamma, None, 0, EPS, "silu", wide, ld))  # in place
        synchronize()
        assert torch.equal(wide[..., :C], y)
        del wide


def test_caller_workspace_gives_the_same_bits():
    for shape in ((2, 8, 8, 64, 8), (3, 70, 64, 64, 8), (2, 9, 9, 40, 4), (1, 5, 5, 2056, 1)):
        p = Norm(*shape)
        need = igc.igc_group_norm_workspace_bytes(*shape)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        before = igc.igc_pool_allocations()
        a, b = p.forward(workspace=ws), p.backward(workspace=ws)
        assert igc.igc_pool_allocations() == before
        if need > 256:
            with pytest.raises(igc.IgcError):
                p.backward(workspace=ws[:need - 256])
        c, d = p.forward(), p.backward()
        synchronize()
        C = shape[3]
        for u, v in zip((*a, *b), (*c, *d)):
            assert torch.equal(u[..., :C], v[..., :C])


def test_captured_calls_replay():
    """Two captured graphs that share one workspace, replayed in turn on new inputs with eager work between."""
    shapes = ((2, 8, 8, 64, 8), (2, 80, 64, 64, 8), (2, 19, 23, 320, 32))
    ws = torch.empty(max(igc.igc_group_norm_workspace_bytes(*s) for s in shapes), dtype=torch.uint8, device="cuda")
    made = []
    for s in shapes:
        p = Norm(*s)
        y, mean, rstd = p.forward(workspace=ws)
        dx, dg, db = p.backward(mean=mean, rstd=rstd, workspace=ws)
        synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            N, H, W, C, G = s
            igc.check(FWD["bf16"](N, H, W, C, G, p.x, p.ld, p.gamma, p.beta, igc.OUT_F32, EPS, p.act, y, p.ld, mean, rstd,
                                  ws))
            igc.check(BWD["bf16"](N, H, W, C, G, p.x, p.ld, p.gamma, p.beta, igc.OUT_F32, mean, rstd, p.act, p.dy, p.ld,
                                  dx, p.ld, dg, db, ws))
        made.append((p, (y, mean, rstd), (dx, dg, db), graph))
    for turn in range(3):
        for p, f, b, graph in made:
            new = Norm(*p.dims, seed=50 + turn)
            for name in ("x", "dy", "gamma", "beta"):
                getattr(p, name).copy_(getattr(new, name))
            for v in (*f, *b):
                v.fill_(float("nan"))
            graph.replay()
            new.check_forward(*f, f"replay {turn}")
            new.check_backward(*b, f"replay {turn}")
            again = new.forward(workspace=ws)
            synchronize()
            assert torch.equal(again[0][..., :p.dims[3]], f[0][..., :p.dims[3]])


def test_gradient_against_differences():
    """loss = sum(dy y): dx, dgamma and dbeta along random directions against central differences in 64 bits."""
    for act in ("silu", "gelu_tanh"):
        p = Norm(2, 5, 6, 24, 4, dtype="fp16", act=act, seed=8)
        N, H, W, C, G = p.dims
        dx, dg, db = p.backward()
        synchronize()
        tol = p.expect_backward()
        at = {"x": p.x[..., :C].double(), "gamma": p.gamma.double(), "beta": p.beta.double()}
        dy = p.dy[..., :C].double()

        def loss(x, gamma, beta):
            v = x.reshape(N, H * W, G, C // G)
            d = v - v.mean((1, 3), keepdim=True)
            xh = (d / torch.sqrt((d * d).mean((1, 3), keepdim=True) + EPS)).reshape(N, H, W, C)
            return (dy * act64(xh * gamma + beta, act)).sum()

        h = 1e-5
        for k, (name, grad) in enumerate((("x", dx[..., :C]), ("gamma", dg), ("beta", db))):
            v = torch.randn(at[name].shape, generator=generator(k), dtype=torch.float64).cuda()
            up, down = dict(at), dict(at)
            up[name], down[name] = at[name] + h * v, at[name] - h * v
            diff = (loss(**up) - loss(**down)) / (2 * h)
            want, e = (u.reshape(v.shape) for u in tol[k])
            bound = ((e + half_step(want, grad.dtype) * 1.01) * v.abs()).sum() + 1e-6 * diff.abs() + 1e-6
            got = (grad.double() * v).sum()
            assert (got - diff).abs() <= bound, (act, name, float(got), float(diff), float(bound))


def test_residual_block():
    """y = x + conv(silu(norm(conv(silu(norm(x))) + b1)) + b2, forward, and its gradients, all through the library; each
    step against the definition in 64 bits of the values the step before stored, and the whole by its chain."""
    N, H, W, C, G, t = 2, 14, 13, 64, 8, torch.bfloat16
    g = generator(77)
    x = normal(g, N, H, W, C, dtype=t).cuda()
    w = [normal(g, C, 3, 3, C, scale=(9 * C) ** -0.5, dtype=t).cuda() for _ in range(2)]
    b = [normal(g, C, scale=0.2).cuda() for _ in range(2)]
    ga, be = [normal(g, C, scale=0.2).cuda() + 1 for _ in range(2)], [normal(g, C, scale=0.2).cuda() for _ in range(2)]
    dy = normal(g, N, H, W, C, dtype=t).cuda()
    geo = (N, H, W, C, C, 3, 3, 1, 1, 1, 1, 1, 1)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    n = [torch.empty_like(x) for _ in range(2)]
    stats = [[torch.empty(N, G, device="cuda") for _ in range(2)] for _ in range(2)]
    h, y = torch.empty_like(x), torch.empty_like(x)

    def norm(k, src):
        igc.check(igc.group_norm_nhwc_bf16_ex(N, H, W, C, G, src, C, ga[k], be[k], igc.OUT_F32, EPS, "silu", n[k], C,
                                              *stats[k], ws))

    norm(0, x)
    igc.check(igc.conv2d_nhwc_implicit_gemm_epilogue_ex(*geo, n[0], w[0], h, igc.OUT_BF16, igc.Epilogue(bias=b[0]), None, ws))
    norm(1, h)
    igc.check(igc.conv2d_nhwc_implicit_gemm_epilogue_ex(*geo, n[1], w[1], y, igc.OUT_BF16,
                                                        igc.Epilogue(bias=b[1], residual=x), None, ws))
    dn, dh, dx = (torch.empty_like(x) for _ in range(3))
    dw, dbias = [torch.empty(C, 3, 3, C, device="cuda") for _ in range(2)], [torch.empty(C, device="cuda") for _ in range(2)]
    dga, dbe = [torch.empty(C, device="cuda") for _ in range(2)], [torch.empty(C, device="cuda") for _ in range(2)]

    def back(k, grad, src, out):
        igc.check(igc.epilogue_backward_bf16_ex(N * H * W, C, "none", grad, C, None, 0, None, 0, dbias[k], igc.OUT_F32, ws))
        igc.check(igc.conv2d_nhwc_wgrad_implicit_gemm_ex(*geo, n[k], grad, dw[k], igc.OUT_F32, None, ws))
        igc.check(igc.conv2d_nhwc_dgrad_implicit_gemm_ex(*geo, grad, w[k], dn, igc.OUT_BF16, None, ws))
        igc.check(igc.group_norm_nhwc_backward_bf16_ex(N, H, W, C, G, src, C, ga[k], be[k], igc.OUT_F32, *stats[k], "silu",
                                                       dn, C, out, C, dga[k], dbe[k], ws))

    back(1, dy, h, dh)
    back(0, dh, x, dx)
    synchronize()
    # the whole in 64 bits; every stored tensor was rounded to bf16 once on the way (h, the norms, dn, dh): each rounding
    # is 2^-8 of a value at most and passes through products whose terms have random signs, so what arrives stays, in
    # the 2-norm, within the sum over the roundings on the longest path (eight, and the gain of 1.5 of what follows each)
    leaves = {k: v.double().requires_grad_() for k, v in
              dict(x=x, w0=w[0], w1=w[1], b0=b[0], b1=b[1], ga0=ga[0], ga1=ga[1], be0=be[0], be1=be[1]).items()}

    def norm64(v, k):
        u = v.reshape(N, H * W, G, C // G)
        d = u - u.mean((1, 3), keepdim=True)
        z = (d / torch.sqrt((d * d).mean((1, 3), keepdim=True) + EPS)).reshape(N, H, W, C) * leaves[f"ga{k}"] + leaves[f"be{k}"]
        return z * torch.sigmoid(z)

    def conv64(v, k):
        cols = torch.nn.functional.unfold(v.permute(0, 3, 1, 2), (3, 3), padding=1).transpose(1, 2)
        out = cols.reshape(-1, 9 * C) @ leaves[f"w{k}"].permute(0, 3, 1, 2).reshape(C, -1).t()
        return out.reshape(N, H, W, C) + leaves[f"b{k}"]

    want = leaves["x"] + conv64(norm64(conv64(norm64(leaves["x"], 0), 0), 1), 1)
    grads = dict(zip(leaves, torch.autograd.grad(want, list(leaves.values()), dy.double())))
    grads["x"] = grads["x"] - dy.double()  # the residual's share, which the caller adds
    got = dict(x=dx, w0=dw[0], w1=dw[1], b0=dbias[0], b1=dbias[1], ga0=dga[0], ga1=dga[1], be0=dbe[0], be1=dbe[1])
    limit = 8 * 1.5 * 2.0 ** -8
    assert float((y.double() - want.detach()).norm() / want.detach().norm()) <= limit
    for k, v in got.items():
        rel = float((v.double() - grads[k]).norm() / grads[k].norm())
        say(f"residual block d{k}: {rel:.2e}")
        assert rel <= limit, (k, rel)


CHUNKED = [
    (1, 40, 33, 2064, 3), (2, 9, 30, 4096, 1), (1, 30, 31, 4120, 5),     # groups across workgroups of 2048 channels
    (2, 30, 31, 264, 264), (1, 33, 30, 2048, 2048), (1, 70, 70, 72, 9),  # one channel a group, and eight
    (7, 56, 9, 736, 1), (12, 21, 15, 1136, 16), (1, 53, 20, 112, 1), (300, 5, 5, 1200, 2), (1, 4, 4, 1280, 1),
    (3, 1, 7, 2048, 32), (2, 1, 7, 2048, 1), (1, 1, 4000, 8, 1), (1, 1, 2049, 8, 1), (1, 1, 3585, 8, 8),
    (1, 2, 33000, 8, 1), (4, 260, 256, 32, 2),
]


@pytest.mark.parametrize("shape", CHUNKED)
def test_chunks_slabs_and_units(shape):
    """Shapes on both sides of one launch and two, of groups in one slab and across several, of one chunk and many."""
    p = Norm(*shape, dtype="bf16", params="f32", act="silu", seed=sum(shape))
    y, mean, rstd = p.forward()
    p.check_forward(y, mean, rstd, f"{shape}")
    p.check_backward(*p.backward(), f"{shape}")
    again = p.forward()
    first, second = p.backward(), p.backward()
    synchronize()
    for a, b in zip((y, mean, rstd) + first, again + second):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), "two runs differ"
    x = p.x.clone()  # in place
    p.check_forward(*p.forward(y=x, x=x), f"{shape} in place")
    dy = p.dy.clone()
    p.check_backward(*p.backward(dx=dy, dy=dy), f"{shape} in place")


@pytest.mark.parametrize("shape", [(2, 32, 32, 2560, 32), (1, 32, 32, 4128, 86), (2, 20, 30, 2072, 7)])
def test_a_group_has_one_result_whichever_slab_it_lies_in(shape):
    """Every group holds the same values, and some lie across two workgroups' channels: the statistics, outputs and
    gradients of all of them are the same to the last bit, on every call."""
    N, H, W, C, G = shape
    g = generator(sum(shape))
    for dtype in ("bf16", "fp16"):
        say(f"slabs {shape} {dtype}")
        one = normal(g, N, H, W, 1, C // G) * 1.5 + normal(g, C // G)
        p = Norm(*shape, dtype=dtype, act="silu", affine=False, x=one.expand(N, H, W, G, C // G).reshape(N, H, W, C))
        p.dy = p.wide(normal(g, N, H, W, 1, C // G, dtype=p.t).expand(N, H, W, G, C // G).reshape(N, H, W, C))
        y, mean, rstd = p.forward()
        p.check_forward(y, mean, rstd, f"{shape}")
        dx, dg, db = p.backward(mean=mean, rstd=rstd)
        p.check_backward(dx, dg, db, f"{shape}")
        for what, v in (("mean", mean), ("rstd", rstd), ("y", p.inside(y, "y").transpose(1, 2).reshape(N, G, -1)),
                        ("dx", p.inside(dx, "dx").transpose(1, 2).reshape(N, G, -1)), ("dgamma", dg.reshape(1, G, -1)),
                        ("dbeta", db.reshape(1, G, -1))):
            assert torch.equal(v, v[:, :1].expand_as(v).contiguous()), f"{what}: groups of equal values differ"
        for _ in range(5):
            again = p.forward()
            grads = p.backward(mean=mean, rstd=rstd)
            synchronize()
            for a, b in zip((y, mean, rstd, dx, dg, db), again + grads):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), "two runs differ"


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_a_constant_group_is_its_beta(dtype):
    """Groups of one value each, in counts that are no powers of two: every sum below is exact in fp32, so the mean is
    the value, the variance 0 and y the rounded beta, to the last bit, in one launch and in chunks."""
    for shape in ((2, 7, 9, 40, 1), (1, 13, 1, 8, 1), (3, 7, 7, 24, 8), (2, 14, 14, 320, 32), (16, 27, 27, 320, 32),
                  (2, 47, 53, 320, 32), (1, 40, 33, 2064, 3)):
        N, H, W, C, G = shape
        for value in (1000.0, 3.0, -7.25):
            say(f"constant {value} {shape} {dtype}")
            p = Norm(*shape, dtype=dtype, act="none", x=torch.full((N, H, W, C), value))
            y, mean, rstd = p.forward()
            p.check_forward(y, mean, rstd, f"constant {value} {shape}")
            assert (mean == value).all()
            assert torch.equal(y[..., :C], p.beta.to(p.t).expand(N, H, W, C))
    p = Norm(2, 14, 14, 320, 32, dtype=dtype)
    x = p.x.clone()
    x[0, 3, 4, 5] = float("inf")
    _, mean, rstd = p.forward(x=x)
    synchronize()
    assert mean[0, 0] == float("inf") and torch.isfinite(mean).sum() == mean.numel() - 1
