"""Timed cases of the fused operators: the matrix product and the convolution with bias, activation and residual in
their epilogue, their gradients, and group norm with an activation over channels-last images.

A case is a dict of plain values.  `prepare` makes its inputs on the GPU from a seed, `run` computes it once -- in
elementary torch operations in 32 bits, or, with `own` set, through the library's entry points -- `exact` computes it
in 64 bits, and `work` counts what the operation has to read, write and compute.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
WORKSPACE_BYTES = 128 << 20  # kept by the program and handed to every call, as a serving or training loop does


def _round8(n):
    return (n + 7) // 8 * 8


# ---- the cases ---------------------------------------------------------------------------------------------------


def listed():
    return [
        # One token through a projection of a decoder: the weights are read once, nothing else counts.
        dict(name="token_1x4096x4096", kind="gemm", M=1, N=4096, K=4096, dtype="bf16", out="bf16", b="col", act="none",
             bias="bf16", residual=True, pre=False),
        # A batch of 17 sequences, one token each, through an up-projection stored K x N.
        dict(name="tokens_17x8192x2048_fp16", kind="gemm", M=17, N=8192, K=2048, dtype="fp16", out="fp16", b="row",
             act="gelu", bias="f32", residual=False, pre=False),
        # The small asymmetric product of the library's own workloads, with everything its epilogue can do.
        dict(name="gemm_128x96x200", kind="gemm", M=128, N=96, K=200, dtype="bf16", out="f32", b="col", act="gelu_tanh",
             bias="f32", residual=True, pre=True),
        # The library's headline product, with the epilogue of a feed-forward layer.
        dict(name="gemm_8192x8192x8192", kind="gemm", M=8192, N=8192, K=8192, dtype="bf16", out="bf16", b="row",
             act="gelu", bias="bf16", residual=True, pre=False),
        # Forward and backward of a feed-forward block over a batch of 4096 tokens.
        dict(name="mlp_train_4096x1024x4096", kind="mlp_train", M=4096, D=1024, F=4096, dtype="bf16", act="gelu_tanh"),
        # Forward and backward of one layer, ragged in every size.
        dict(name="linear_train_777x1336x520_fp16", kind="linear_train", M=777, N=1336, K=520, dtype="fp16", act="silu"),
        # The library's 3 x 3 convolution as the second half of a residual block.
        dict(name="conv_n32_56x56_c256_k256_3x3", kind="conv", N=32, H=56, W=56, C=256, K=256, R=3, S=3, stride=1, pad=1,
             dtype="bf16", act="none", residual=True),
        # An odd image size, bias and activation only.
        dict(name="conv_n16_27x27_c256_k256_3x3", kind="conv", N=16, H=27, W=27, C=256, K=256, R=3, S=3, stride=1, pad=1,
             dtype="fp16", act="relu", residual=False),
        # The deepest, smallest images of a generator at a batch of two: launch latency.
        dict(name="gn_n2_8x8_c1280", kind="gn", N=2, H=8, W=8, C=1280, G=32, dtype="bf16", params="f32", act="silu"),
        # The input of the 3 x 3 convolution above.
        dict(name="gn_n32_56x56_c256", kind="gn", N=32, H=56, W=56, C=256, G=32, dtype="bf16", params="bf16", act="silu"),
        # The same in training: statistics kept, all three gradients.
        dict(name="gn_train_n32_56x56_c256", kind="gn_train", N=32, H=56, W=56, C=256, G=32, dtype="bf16", params="f32",
             act="silu"),
        # Groups of ten channels, which no vector load fits, on odd images.
        dict(name="gn_train_n16_27x27_c320_fp16", kind="gn_train", N=16, H=27, W=27, C=320, G=32, dtype="fp16",
             params="f32", act="none"),
    ]


ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("token", "gemm", "mlp_train", "linear_train", "conv", "gn", "gn_train"))
    dtype = rng.choice(("bf16", "fp16"))
    # the derivative of relu jumps at zero, where a sum's last bit decides: gradients are drawn with the smooth ones
    act = rng.choice([a for a in ACTS if a != "relu" or "train" not in kind])
    if kind == "token":
        return dict(kind="gemm", M=_log_int(rng, 1, 64), N=_log_int(rng, 256, 16384), K=_log_int(rng, 256, 16384),
                    dtype=dtype, out=dtype, b=rng.choice(("row", "col")), act=act, bias=rng.choice((dtype, "f32")),
                    residual=rng.random() < 0.5, pre=False)
    if kind == "gemm":
        K = _log_int(rng, 64, 8192)
        out = rng.choice((dtype, dtype, "f32")) if K <= 4096 else dtype
        return dict(kind="gemm", M=_log_int(rng, 65, 8192), N=_log_int(rng, 64, 8192), K=K, dtype=dtype, out=out,
                    b=rng.choice(("row", "col")), act=act, bias=rng.choice((dtype, "f32")),
                    residual=rng.random() < 0.5, pre=rng.random() < 0.3)
    if kind == "mlp_train":
        return dict(kind=kind, M=_log_int(rng, 64, 4096), D=_log_int(rng, 64, 2048), F=_log_int(rng, 128, 8192),
                    dtype=dtype, act=act)
    if kind == "linear_train":
        return dict(kind=kind, M=_log_int(rng, 64, 8192), N=_log_int(rng, 64, 4096), K=_log_int(rng, 64, 4096),
                    dtype=dtype, act=act)
    if kind == "conv":
        r = rng.choice((1, 3))
        return dict(kind=kind, N=_log_int(rng, 1, 32), H=rng.randint(7, 64), W=rng.randint(7, 64),
                    C=8 * _log_int(rng, 4, 48), K=8 * _log_int(rng, 4, 48), R=r, S=r, stride=rng.choice((1, 1, 2)),
                    pad=r // 2, dtype=dtype, act=act, residual=rng.random() < 0.5)
    C = 8 * _log_int(rng, 4, 160)
    G = rng.choice([g for g in (1, 2, 4, 8, 16, 32, 64) if C % g == 0])
    return dict(kind=kind, N=_log_int(rng, 1, 32), H=rng.randint(4, 64), W=rng.randint(4, 64), C=C, G=G, dtype=dtype,
                params=rng.choice((dtype, "f32")), act=act)


# ---- inputs ------------------------------------------------------------------------------------------------------


class _Maker:
    """Seeded normal values on the GPU, rounded once to their type, in rows of a 16-byte multiple."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.g, device="cuda") * scale).to(dtype)

    def matrix(self, rows, cols, scale, dtype):
        return self.normal(rows, _round8(cols), scale=scale, dtype=dtype)[:, :cols]


def _out_size(c):
    return ((c["H"] + 2 * c["pad"] - c["R"]) // c["stride"] + 1, (c["W"] + 2 * c["pad"] - c["S"]) // c["stride"] + 1)


def prepare(case, seed):
    c, m = case, _Maker(seed)
    t = DTYPES[c["dtype"]]
    s = dict(c, workspace=torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda"))
    if c["kind"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        s["A"] = m.matrix(M, K, 1.0, t)
        s["B"] = m.matrix(N, K, K ** -0.5, t) if c["b"] == "col" else m.matrix(K, N, K ** -0.5, t)
        s["bias_values"] = m.normal(N, scale=0.5, dtype=DTYPES[c["bias"]])
        if c["residual"]:
            s["res"] = m.matrix(M, N, 1.0, t)
    elif c["kind"] == "linear_train":
        M, N, K = c["M"], c["N"], c["K"]
        s["x"], s["w"] = m.matrix(M, K, 1.0, t), m.matrix(N, K, K ** -0.5, t)
        s["b"], s["dy"] = m.normal(N, scale=0.5, dtype=t), m.matrix(M, N, 1.0, t)
    elif c["kind"] == "mlp_train":
        M, D, F = c["M"], c["D"], c["F"]
        s["x"] = m.matrix(M, D, 1.0, t)
        s["w1"], s["b1"] = m.matrix(F, D, D ** -0.5, t), m.normal(F, scale=0.5, dtype=t)
        s["w2"], s["b2"] = m.matrix(D, F, F ** -0.5, t), m.normal(D, scale=0.5, dtype=t)
        s["dy"] = m.matrix(M, D, 1.0, t)
    elif c["kind"] == "conv":
        P, Q = _out_size(c)
        s["x"] = m.normal(c["N"], c["H"], c["W"], c["C"], dtype=t)
        s["w"] = m.normal(c["K"], c["R"], c["S"], c["C"], scale=(c["R"] * c["S"] * c["C"]) ** -0.5, dtype=t)
        s["bias_values"] = m.normal(c["K"], scale=0.5)
        if c["residual"]:
            s["res"] = m.normal(c["N"], P, Q, c["K"], dtype=t)
    else:
        # activations of a network: every channel has its own mean and width
        C, p = c["C"], DTYPES[c["params"]]
        centre, width = m.normal(C), 0.5 + m.normal(C).abs()
        s["x"] = (m.normal(c["N"], c["H"], c["W"], C) * width + centre).to(t)
        s["gamma"], s["beta"] = (1 + m.normal(C, scale=0.2)).to(p), m.normal(C, scale=0.2, dtype=p)
        if c["kind"] == "gn_train":
            s["dy"] = m.normal(c["N"], c["H"], c["W"], C, dtype=t)
    return s


# ---- plain forms: elementary operations in 32 bits, rounded once --------------------------------------------------

SQRT_HALF = math.sqrt(0.5)
GELU_C, GELU_A = math.sqrt(2 / math.pi), 0.044715
EPS = 1e-5


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * SQRT_HALF))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(GELU_C * (z + GELU_A * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * SQRT_HALF)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(GELU_C * (z + GELU_A * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * GELU_C * (1 + 3 * GELU_A * z * z)
    if act == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    return torch.ones_like(z)


def _plain_gemm(s):
    A, B = s["A"].float(), s["B"].float()
    z = A @ (B.t() if s["b"] == "col" else B) + s["bias_values"].float()
    y = _act(z, s["act"])
    if s["residual"]:
        y = y + s["res"].float()
    y = y.to(DTYPES[s["out"]])
    return {"y": y, "pre": z.to(DTYPES[s["dtype"]])} if s["pre"] else {"y": y}


def _plain_linear_train(s):
    t = DTYPES[s["dtype"]]
    x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
    z = x @ w.t() + s["b"].float()
    dz = dy * _act_grad(z, s["act"])
    return {"y": _act(z, s["act"]).to(t), "dx": (dz @ w).to(t), "dw": (dz.t() @ x).to(t), "db": dz.sum(0).to(t)}


def _plain_mlp_train(s):
    t = DTYPES[s["dtype"]]
    x, w1, w2, dy = s["x"].float(), s["w1"].float(), s["w2"].float(), s["dy"].float()
    z = x @ w1.t() + s["b1"].float()
    h = _act(z, s["act"])
    y = h @ w2.t() + s["b2"].float() + x
    dz = (dy @ w2) * _act_grad(z, s["act"])
    return {"y": y.to(t), "dx": (dz @ w1 + dy).to(t), "dw1": (dz.t() @ x).to(t), "db1": dz.sum(0).to(t),
            "dw2": (dy.t() @ h).to(t), "db2": dy.sum(0).to(t)}


def _plain_conv(s):
    N, H, W, C, K, R, S, st, pad = (s[k] for k in ("N", "H", "W", "C", "K", "R", "S", "stride", "pad"))
    P, Q = _out_size(s)
    x = torch.zeros(N, H + 2 * pad, W + 2 * pad, C, device="cuda")
    x[:, pad:pad + H, pad:pad + W] = s["x"].float()
    a, b, e, _ = x.stride()
    windows = x.as_strided((N, P, Q, R, S, C), (a, st * b, st * e, b, e, 1)).reshape(N * P * Q, R * S * C)
    z = windows @ s["w"].float().reshape(K, R * S * C).t() + s["bias_values"]
    y = _act(z, s["act"]).reshape(N, P, Q, K)
    if s["residual"]:
        y = y + s["res"].float()
    return {"y": y.to(DTYPES[s["dtype"]])}


def _plain_gn(s):
    N, H, W, C, G = (s[k] for k in ("N", "H", "W", "C", "G"))
    t = DTYPES[s["dtype"]]
    x = s["x"].float().reshape(N, H * W, G, C // G)
    mean = x.mean((1, 3), keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean((1, 3), keepdim=True) + EPS)
    xh = d * rstd
    gamma, beta = s["gamma"].float().reshape(G, C // G), s["beta"].float().reshape(G, C // G)
    z = xh * gamma + beta
    y = _act(z, s["act"]).reshape(N, H, W, C).to(t)
    if s["kind"] == "gn":
        return {"y": y}
    dz = s["dy"].float().reshape(N, H * W, G, C // G) * _act_grad(z, s["act"])
    p = DTYPES[s["params"]]
    dxh = dz * gamma
    dx = rstd * (dxh - dxh.mean((1, 3), keepdim=True) - xh * (dxh * xh).mean((1, 3), keepdim=True))
    return {"y": y, "mean": mean.reshape(N, G), "rstd": rstd.reshape(N, G), "dx": dx.reshape(N, H, W, C).to(t),
            "dgamma": (dz * xh).sum((0, 1)).reshape(C).to(p), "dbeta": dz.sum((0, 1)).reshape(C).to(p)}


# ---- the library's calls ------------------------------------------------------------------------------------------


def _rows(rows, cols, dtype):
    """An output of rows x cols whose rows are a 16-byte multiple apart."""
    return torch.empty(rows, _round8(cols), dtype=dtype, device="cuda")[:, :cols]


def _gemm(igc, dtype, A, la, B, lb, D, epi, ws):
    """D = epilogue(A * B); a column-major operand is given as its transpose, the way it lies in memory."""
    M, N = D.shape
    K = A.shape[1] if la == igc.ROW_MAJOR else A.shape[0]
    out = igc.out_code(D.dtype)
    if epi is None:
        f = igc.gemm_bf16_ex if dtype == "bf16" else igc.gemm_fp16_ex
        igc.check(f(M, N, K, A, A.stride(0), la, B, B.stride(0), lb, D, D.stride(0), out, workspace=ws))
    else:
        f = igc.gemm_bf16_epilogue_ex if dtype == "bf16" else igc.gemm_fp16_epilogue_ex
        igc.check(f(M, N, K, A, A.stride(0), la, B, B.stride(0), lb, D, D.stride(0), out, epi, workspace=ws))
    return D


def _own_gemm(igc, s):
    D = _rows(s["M"], s["N"], DTYPES[s["out"]])
    pre = _rows(s["M"], s["N"], DTYPES[s["dtype"]]) if s["pre"] else None
    epi = igc.Epilogue(act=s["act"], bias=s["bias_values"], residual=s["res"] if s["residual"] else None, pre=pre)
    _gemm(igc, s["dtype"], s["A"], igc.ROW_MAJOR, s["B"], igc.COL_MAJOR if s["b"] == "col" else igc.ROW_MAJOR, D, epi,
          s["workspace"])
    return {"y": D, "pre": pre} if s["pre"] else {"y": D}


def _own_linear_train(igc, s):
    M, N, K, d, ws = s["M"], s["N"], s["K"], s["dtype"], s["workspace"]
    t, row, col = DTYPES[d], igc.ROW_MAJOR, igc.COL_MAJOR
    pre, dz, db = _rows(M, N, t), _rows(M, N, t), torch.empty(N, dtype=t, device="cuda")
    y = _gemm(igc, d, s["x"], row, s["w"], col, _rows(M, N, t), igc.Epilogue(act=s["act"], bias=s["b"], pre=pre), ws)
    back = igc.epilogue_backward_bf16_ex if d == "bf16" else igc.epilogue_backward_fp16_ex
    igc.check(back(M, N, s["act"], s["dy"], s["dy"].stride(0), pre, pre.stride(0), dz, dz.stride(0), db,
                   igc.out_code(t), workspace=ws))
    dx = _gemm(igc, d, dz, row, s["w"], row, _rows(M, K, t), None, ws)
    dw = _gemm(igc, d, dz, col, s["x"], row, _rows(N, K, t), None, ws)
    return {"y": y, "dx": dx, "dw": dw, "db": db}


def _own_mlp_train(igc, s):
    M, D, F, d, ws = s["M"], s["D"], s["F"], s["dtype"], s["workspace"]
    t, row, col = DTYPES[d], igc.ROW_MAJOR, igc.COL_MAJOR
    pre, db1, db2 = _rows(M, F, t), torch.empty(F, dtype=t, device="cuda"), torch.empty(D, dtype=t, device="cuda")
    h = _gemm(igc, d, s["x"], row, s["w1"], col, _rows(M, F, t), igc.Epilogue(act=s["act"], bias=s["b1"], pre=pre), ws)
    y = _gemm(igc, d, h, row, s["w2"], col, _rows(M, D, t), igc.Epilogue(bias=s["b2"], residual=s["x"]), ws)
    back = igc.epilogue_backward_bf16_ex if d == "bf16" else igc.epilogue_backward_fp16_ex
    code = igc.out_code(t)
    igc.check(back(M, D, "none", s["dy"], s["dy"].stride(0), None, 0, None, 0, db2, code, workspace=ws))
    dz = _gemm(igc, d, s["dy"], row, s["w2"], row, _rows(M, F, t), igc.Epilogue(act=s["act"], pre=pre, backward=True), ws)
    igc.check(back(M, F, "none", dz, dz.stride(0), None, 0, None, 0, db1, code, workspace=ws))
    dx = _gemm(igc, d, dz, row, s["w1"], row, _rows(M, D, t), igc.Epilogue(residual=s["dy"]), ws)
    dw1 = _gemm(igc, d, dz, col, s["x"], row, _rows(F, D, t), None, ws)
    dw2 = _gemm(igc, d, s["dy"], col, h, row, _rows(D, F, t), None, ws)
    return {"y": y, "dx": dx, "dw1": dw1, "db1": db1, "dw2": dw2, "db2": db2}


def _own_conv(igc, s):
    P, Q = _out_size(s)
    y = torch.empty(s["N"], P, Q, s["K"], dtype=DTYPES[s["dtype"]], device="cuda")
    epi = igc.Epilogue(act=s["act"], bias=s["bias_values"], residual=s["res"] if s["residual"] else None)
    f = igc.conv2d_nhwc_implicit_gemm_epilogue_ex if s["dtype"] == "bf16" else \
        igc.conv2d_nhwc_implicit_gemm_epilogue_fp16_ex
    igc.check(f(s["N"], s["H"], s["W"], s["C"], s["K"], s["R"], s["S"], s["stride"], s["stride"], s["pad"], s["pad"], 1,
                1, s["x"], s["w"], y, igc.out_code(y.dtype), epi, workspace=s["workspace"]))
    return {"y": y}


def _own_gn(igc, s):
    N, H, W, C, G, x, ws = (s[k] for k in ("N", "H", "W", "C", "G", "x", "workspace"))
    bf16, train, p = s["dtype"] == "bf16", s["kind"] == "gn_train", igc.out_code(s["gamma"].dtype)
    y = torch.empty_like(x)
    mean = torch.empty(N, G, device="cuda") if train else None
    rstd = torch.empty(N, G, device="cuda") if train else None
    f = igc.group_norm_nhwc_bf16_ex if bf16 else igc.group_norm_nhwc_fp16_ex
    igc.check(f(N, H, W, C, G, x, C, s["gamma"], s["beta"], p, EPS, s["act"], y, C, mean, rstd, workspace=ws))
    if not train:
        return {"y": y}
    dx, dgamma, dbeta = torch.empty_like(x), torch.empty_like(s["gamma"]), torch.empty_like(s["beta"])
    f = igc.group_norm_nhwc_backward_bf16_ex if bf16 else igc.group_norm_nhwc_backward_fp16_ex
    igc.check(f(N, H, W, C, G, x, C, s["gamma"], s["beta"], p, mean, rstd, s["act"], s["dy"], C, dx, C, dgamma, dbeta,
                workspace=ws))
    return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def run(state):
    kind = state["kind"]
    if own:
        import implicit_gemm_conv_amd as igc
        return {"gemm": _own_gemm, "linear_train": _own_linear_train, "mlp_train": _own_mlp_train, "conv": _own_conv,
                "gn": _own_gn, "gn_train": _own_gn}[kind](igc, state)
    return {"gemm": _plain_gemm, "linear_train": _plain_linear_train, "mlp_train": _plain_mlp_train,
            "conv": _plain_conv, "gn": _plain_gn, "gn_train": _plain_gn}[kind](state)


# ---- what an operation cannot do without ---------------------------------------------------------------------------


def work(case):
    c = case
    e = 2  # bytes of a 16-bit value
    size = {"bf16": 2, "fp16": 2, "f32": 4}
    if c["kind"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": (M * K + K * N) * e + N * size[c["bias"]] + M * N * (size[c["out"]] + e * c["residual"] + e * c["pre"]),
                "flops": 2 * M * N * K}
    if c["kind"] == "linear_train":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": (M * K + N * K + N + M * N) * e + (M * N + M * K + N * K + N) * e, "flops": 6 * M * N * K}
    if c["kind"] == "mlp_train":
        M, D, F = c["M"], c["D"], c["F"]
        weights = 2 * D * F + D + F
        return {"bytes": (2 * M * D + weights) * e + (2 * M * D + weights) * e, "flops": 12 * M * D * F}
    if c["kind"] == "conv":
        P, Q = _out_size(c)
        k, out = c["R"] * c["S"] * c["C"], c["N"] * P * Q * c["K"]
        return {"bytes": (c["N"] * c["H"] * c["W"] * c["C"] + c["K"] * k + out * (1 + c["residual"])) * e + 4 * c["K"],
                "flops": 2 * out * k}
    n, params, stats = c["N"] * c["H"] * c["W"] * c["C"], c["C"] * size[c["params"]], c["N"] * c["G"] * 4
    if c["kind"] == "gn":
        return {"bytes": 2 * n * e + 2 * params, "flops": 10 * n}
    return {"bytes": 4 * n * e + 4 * params + 2 * stats, "flops": 30 * n}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------


def _activate64(z, act):
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: z * 0.5 * torch.erfc(-z / 2 ** 0.5),
            # 0.5 (1 + tanh u) = sigmoid(2 u)
            "gelu_tanh": lambda: z * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3))}[act]()


def exact(case, seed):
    s, kind = prepare(case, seed), case["kind"]
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    if kind == "gemm":
        z = torch.addmm(d["bias_values"], d["A"], d["B"].T if case["b"] == "col" else d["B"])
        y = _activate64(z, case["act"])
        if case["residual"]:
            y += d["res"]
        return {"y": y, "pre": z} if case["pre"] else {"y": y}
    if kind == "conv":
        w = d["w"].permute(0, 3, 1, 2).reshape(case["K"], -1)
        P, Q = _out_size(case)
        images = []
        for image in d["x"]:
            cols = torch.nn.functional.unfold(image.permute(2, 0, 1)[None], (case["R"], case["S"]), padding=case["pad"],
                                              stride=case["stride"])[0]
            images.append((w @ cols).T.reshape(P, Q, case["K"]))
        y = _activate64(torch.stack(images) + d["bias_values"], case["act"])
        return {"y": y + d["res"] if case["residual"] else y}
    if kind in ("linear_train", "mlp_train"):
        names = ("x", "w", "b") if kind == "linear_train" else ("x", "w1", "b1", "w2", "b2")
        leaf = {n: d[n].requires_grad_() for n in names}
        if kind == "linear_train":
            y = _activate64(leaf["x"] @ leaf["w"].T + leaf["b"], case["act"])
        else:
            h = _activate64(leaf["x"] @ leaf["w1"].T + leaf["b1"], case["act"])
            y = h @ leaf["w2"].T + leaf["b2"] + leaf["x"]
        grads = dict(zip(names, torch.autograd.grad(y, [leaf[n] for n in names], d["dy"])))
        order = ("x", "w", "b") if kind == "linear_train" else ("x", "w1", "b1", "w2", "b2")
        return {"y": y.detach(), **{"d" + n: grads[n] for n in order}}
    N, C, G = case["N"], case["C"], case["G"]
    x, gamma, beta = d["x"].requires_grad_(), d["gamma"].requires_grad_(), d["beta"].requires_grad_()
    g = x.reshape(N, -1, G, C // G).transpose(1, 2).reshape(N, G, -1)
    var, mean = torch.var_mean(g, -1, correction=0, keepdim=True)
    rstd = (var + EPS).rsqrt()
    xh = ((g - mean) * rstd).reshape(N, G, -1, C // G).transpose(1, 2).reshape(x.shape)
    y = _activate64(xh * gamma + beta, case["act"])
    if kind == "gn":
        return {"y": y.detach()}
    dx, dgamma, dbeta = torch.autograd.grad(y, (x, gamma, beta), d["dy"])
    return {"y": y.detach(), "mean": mean.detach().reshape(N, G), "rstd": rstd.detach().reshape(N, G), "dx": dx,
            "dgamma": dgamma, "dbeta": dbeta}
