"""Definitions in 64 bits of the fused operators, and the tolerances their tests use.

Half a step of rounding to a type is finfo(t).eps / 2 of the value (below the smallest normal number, half its lowest
step).  The kernels compute in fp32; what that may be off by is derived where it is used, from
  - a sum of n products a*b in any order: n * 2^-24 * sum |a b|;
  - the activations, evaluated with the hardware's exp2 and reciprocal (about 2^-23 each): the argument of exp2 is
    rounded once or twice, which moves the result by up to z^2 * 2^-23 of itself; ACT_REL * (1 + z^2) covers both,
    and the 8.6e-7 of the fitted tail of gelu;
  - |act'| <= 1.13 and |act''| <= 1.2 for every activation but relu at 0.
"""
import math

import torch

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "f16": torch.float16, "f32": torch.float32}
U32 = 2.0 ** -24
ACT_REL = 2.0 ** -19
ACT_LIP, ACT_CURVE = 1.13, 1.2
GRAD_ABS = 2.0 ** -18  # act' is a sum of terms of at most about 1.2 in size, each off by a few 2^-20


def act64(z, act):
    if act == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), z)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def act_grad64(z, act):
    if act == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), torch.where(z > 0, torch.ones_like(z), z))
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        s = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return s + z * s * (1 - s) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def half_step(y, dtype):
    """Half a step of `dtype` at the magnitude of y (float64)."""
    f = torch.finfo(dtype)
    return torch.clamp(y.abs(), min=f.tiny) * (f.eps / 2)


def assert_within(got, want, tol, what=""):
    """|got - want| <= tol + half a step of got's type, element by element; want and tol are float64."""
    assert got.shape == want.shape, (what, got.shape, want.shape)
    g = got.double()
    bound = tol + half_step(torch.maximum(want.abs(), want.abs() + tol), got.dtype)
    off = (g - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = int(torch.argmax(torch.where(bad, torch.nan_to_num(off / bound, nan=float("inf")), torch.zeros_like(off))))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; worst at flat {i}: got "
                             f"{g.flatten()[i].item()!r} want {want.flatten()[i].item()!r} bound "
                             f"{bound.flatten()[i].item()!r}")
    return float((off / bound).max()) if off.numel() else 0.0


def generator(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def padded(t, ld, poison=float("nan"), extra_rows=0):
    """t (rows x cols) on the GPU in rows ld apart, NaN in the padding and in `extra_rows` rows after the last:
    (view, whole storage)."""
    rows, cols = t.shape
    buf = torch.full((rows + extra_rows, ld), poison, dtype=t.dtype)
    buf[:rows, :cols] = t
    buf = buf.cuda()
    return buf[:rows, :cols], buf


def round8(n):
    return (n + 7) // 8 * 8
