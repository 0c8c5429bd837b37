"""Row operators (RMS norm to 16 and 8 bits, its gradient, rows to 8 bits) where their forms cross: every type and address
of gamma with every remainder of a row's length by 8, gradients whose sums are exact, rows at the ends of the number range.
Definitions and tolerances are those of test_int8_ops_gpu.py unless a test says otherwise."""
import pytest
import torch

import implicit_gemm_conv_amd as igc
from fused_util import DT, U32, generator, padded, round8
from gpu_util import synchronize
from test_int8_ops_gpu import BACK, EPS, NORM8, Norm, check_int8, up16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    igc.lib()


def place(v, odd):
    """A view of v's values at a 16-byte multiple, or one value past it, with NaN before and after them."""
    buf = torch.full((v.numel() + 16,), float("nan"), dtype=v.dtype, device="cuda")
    at = 16 // v.element_size() + odd
    out = buf[at:at + v.numel()]
    out.copy_(v)
    assert (out.data_ptr() % 16 == 0) == (not odd)
    return out


@pytest.mark.parametrize("gamma", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("C", [1, 2, 3, 5, 6, 7, 9, 61, 131, 413, 1006, 1535, 2051, 4101, 8195, 16389, 20003, 32773])
def test_gamma_of_every_type_and_address(C, odd, gamma):
    """NaN lies around gamma: a value that is not gamma's own would reach the largest magnitude and the gradient's sums."""
    for M, dtype, residual, dh in ((3, "bf16", True, False), (3, "fp16", False, True)):
        n = Norm(M, C, dtype, residual=residual, gamma=gamma, seed=C)
        n.gamma = place(n.gamma, odd)
        what = f"{M}x{C} {dtype} gamma {gamma} odd {odd}"
        y, h, rstd, scale = n.out(), n.out(), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        n.forward(y, h, rstd)
        n.check(y, h, rstd, what)
        qbuf = torch.full((M + 2, up16(C) + 16), 99, dtype=torch.int8, device="cuda")
        a, b = n.args()
        igc.check(NORM8[dtype](M, C, *a, None, 0, *b, qbuf, qbuf.stride(0), scale))
        synchronize()
        check_int8(qbuf[:M, :C], qbuf, scale, n.y, n.rstd_rel + 2 * U32, what)
        dgamma, dx = place(torch.zeros(C, dtype=DT[gamma]), odd), n.out()
        n.backward(dx, dgamma, dh)
        n.check_backward(dx, dgamma, dh, what)


POWERS = [0, 62, 90, 110, -40, -60, -75, -100, -115]


@pytest.mark.parametrize("eps", [EPS, 0.0])
@pytest.mark.parametrize("C", [60, 400, 1000, 2000, 5000, 16384, 20000, 40000])
def test_norm_of_every_magnitude(C, eps):
    """Rows whose squares leave fp32's range though their root mean square does not, beside ordinary ones: each is normed as
    any other, forward, to 8 bits and back."""
    M = 3 * len(POWERS)
    n = Norm(M, C, "bf16", residual=C % 16 == 0, seed=C)
    scale2 = torch.tensor(POWERS * 3, dtype=torch.float32, device="cuda").exp2()[:, None]
    n.x.copy_(n.x.float() * scale2)
    if n.res is not None:
        n.res.copy_(n.res.float() * scale2)
    n.define()
    hd = n.h.double()
    n.rstd = 1 / torch.sqrt((hd * hd).mean(1) + eps)
    n.y = hd * n.rstd[:, None] * n.g64
    a, _ = n.args()
    y, rstd = n.out(), torch.empty(M, device="cuda")
    igc.check(igc.rms_norm_bf16(M, C, *a, None, 0, n.gamma, igc.OUT_F32, eps, y, n.ld, rstd))
    n.check(y, None, rstd, f"eps {eps}")
    qbuf, scale = torch.full((M + 2, up16(C) + 16), 99, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    igc.check(igc.rms_norm_int8_bf16(M, C, *a, None, 0, n.gamma, igc.OUT_F32, eps, qbuf, qbuf.stride(0), scale))
    synchronize()
    check_int8(qbuf[:M, :C], qbuf, scale, n.y, n.rstd_rel + 2 * U32, f"eps {eps} to 8 bits")
    dx, dgamma = n.out(), torch.empty(C, device="cuda")
    n.backward(dx, dgamma, dh=False, rstd=rstd)
    n.check_backward(dx, dgamma, dh=False, what=f"eps {eps}")


def norm_to_8_bits(n, x, gamma):
    """(q, scale) of rows x with n's sizes."""
    qbuf, scale = torch.full((n.M, up16(n.C)), 99, dtype=torch.int8, device="cuda"), torch.zeros(n.M, device="cuda")
    igc.check(NORM8[n.dtype](n.M, n.C, x, n.ld, None, 0, None, 0, gamma, igc.OUT_F32, EPS, qbuf, up16(n.C), scale))
    synchronize()
    assert (qbuf[:, n.C:] == 99).all()
    return qbuf[:, :n.C], scale


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("C", [60, 1000, 4096, 40000])
def test_rows_to_8_bits_without_a_largest_value(C, dtype):
    """An infinity or a NaN in gamma, or an h * gamma that passes fp32: scale NaN and zeros, so that a product of the row is
    NaN.  A row of zeros meets 0 * infinity, but not a gamma that is merely large."""
    n = Norm(5, C, dtype, residual=False, gamma="f32", seed=C)
    n.x[1] = 0
    for g in (float("inf"), float("-inf"), float("nan")):
        gamma = n.gamma.clone()
        gamma[C // 2] = g
        q, scale = norm_to_8_bits(n, n.xbuf, gamma)
        assert torch.isnan(scale).all() and (q == 0).all(), (g, scale, q.unique())
    gamma, x = n.gamma.clone(), n.xbuf.clone()
    gamma[C // 2], x[:, C // 2] = 1e38, 50
    x[1] = 0
    q, scale = norm_to_8_bits(n, x, gamma)
    assert torch.isnan(scale[[0, 2, 3, 4]]).all() and scale[1] == 0 and (q == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("C", [60, 1000, 4096, 40000])
def test_nan_of_gamma_gives_zeros_in_8_bits(C, dtype):
    """Whatever a NaN's sign and low bits."""
    n = Norm(5, C, dtype, residual=False, gamma="f32", seed=C)
    gamma = n.gamma.clone()
    gamma[C // 2:C // 2 + 5] = torch.tensor([0x7FC00000, 0x7FC00001, 0x7FFFFFFF, -1, 0x7F80007F],
                                            dtype=torch.int32).view(torch.float32).cuda()
    q, scale = norm_to_8_bits(n, n.xbuf, gamma)
    assert torch.isnan(scale).all() and (q == 0).all(), q.unique()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,C", [(1, 72), (7, 72), (17, 72), (4111, 72), (20011, 72), (33, 300), (9001, 300), (3, 700),
                                 (4099, 700), (3001, 1500), (1601, 4000), (1031, 8000), (1029, 16000), (777, 20000),
                                 (261, 40000), (1, 40000)])
def test_norm_gradient_sums_every_row_once(M, C, dtype):
    """With whole numbers and rstd 1 every sum for dgamma is exact: rows in several turns of a workgroup, the last of them
    part of one, each count once.  NaN lies behind the last row and each row's end."""
    g, t = generator(M + C), DT[dtype]
    ld = round8(C) + 8
    h, hbuf = padded(torch.randint(-3, 4, (M, C), generator=g).to(t), ld, extra_rows=16)
    dy, dybuf = padded(torch.randint(-3, 4, (M, C), generator=g).to(t), ld, extra_rows=16)
    rstd = torch.full((M + 16,), float("nan"), device="cuda")
    rstd[:M] = 1
    want = (h.double() * dy.double()).sum(0)
    for out in (torch.float32, torch.bfloat16):
        dx, dgamma = torch.empty(M, ld, dtype=t, device="cuda"), torch.full((C + 8,), 99, dtype=out, device="cuda")
        igc.check(BACK[dtype](M, C, hbuf, ld, None, igc.out_code(out), rstd, dybuf, ld, None, 0, dx, ld, dgamma))
        synchronize()
        assert torch.equal(dgamma[:C], want.float().to(out)) and (dgamma[C:] == 99).all()
