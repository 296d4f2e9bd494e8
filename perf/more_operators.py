"""Measured cases of a mixture-of-experts block's operators in 8 and 4 bits.

Three operators:

* root-mean-square norm ("rms_fwd", "rms_bwd"): the addition of a sublayer's
  output to the residual stream and the norm of the sum, with its output as
  BF16 and/or as an FP8 GEMM operand and the normalised rows as an 8-bit
  checkpoint; the backward pass from the stream or from that checkpoint, with
  the gradient that arrives along the stream and the reduction of gamma's;
* products grouped by expert ("moe_fprop", "moe_dgrad", "moe_wgrad"): rows
  sorted by expert times each expert's weights, with segments that only the
  device knows, and both gradients;
* 4-bit floating point in blocks of 32 with E8M0 scales ("fp4_cast",
  "fp4_gemm"): the cast along rows, and along columns too for the backward
  products, brought back; products of 4-bit weights with 8- or 4-bit rows.

``own`` selects the side: False, the formulas in elementary torch operations
in 32 bits; True, the calls of ``scaled_fp8_gemm_amd.fp8sg``.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
EPS = 1e-5
FLT_MAX = torch.finfo(torch.float32).max
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# 8-bit formats: torch's type, largest value, largest value = 1.75 * 2^P
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0, "e2m1": 6.0}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step's rows: latency
        {"name": "rms_fwd 8x4096", "op": "rms_fwd", "rows": 8, "cols": 4096, "x": "bf16",
         "w": "bf16", "delta": True, "y": True, "yq": "none", "ckpt": False},
        # the norm in front of the GPT-175B share's MXFP8 GEMM, FP32 residual
        # stream, FP8 operand and 8-bit checkpoint
        {"name": "rms_fwd 4096x12288 f32 mx ckpt", "op": "rms_fwd", "rows": 4096, "cols": 12288,
         "x": "f32", "w": "f32", "delta": True, "y": False, "yq": "mx", "ckpt": True},
        # training at the 13B width: backward from the 8-bit checkpoint
        {"name": "rms_bwd 8192x5120 ckpt", "op": "rms_bwd", "rows": 8192, "cols": 5120,
         "x": "bf16", "w": "f32", "ckpt": True, "dres": True},
        # an FP32 stream of an odd width
        {"name": "rms_bwd 1000x1003 f32", "op": "rms_bwd", "rows": 1000, "cols": 1003,
         "x": "f32", "w": "bf16", "ckpt": False, "dres": True},
        # one expert-parallel rank's tokens through 8 experts of the 7B MLP's
        # width, blockwise recipe
        {"name": "moe_fprop 8192 e8k2 block", "op": "moe_fprop", "tokens": 8192, "k": 2,
         "experts": 8, "inn": 4096, "out": 11008, "scaling": "block", "fa": "e4m3",
         "fb": "e4m3", "pad": 128},
        # the weight gradients of that, MX recipe
        {"name": "moe_wgrad 8192 e8k2 mx", "op": "moe_wgrad", "tokens": 8192, "k": 2,
         "experts": 8, "inn": 4096, "out": 11008, "scaling": "mx", "fa": "e4m3", "fb": "e4m3",
         "pad": 128},
        # fine-grained experts with short ragged segments, per-tensor scales,
        # gradient rows in E5M2
        {"name": "moe_dgrad 1000 e64k6 tensor", "op": "moe_dgrad", "tokens": 1000, "k": 6,
         "experts": 64, "inn": 1408, "out": 2000, "scaling": "tensor", "fa": "e5m2",
         "fb": "e4m3", "pad": 16},
        # a decode step's tokens through 8 experts with 4-bit weights
        {"name": "moe_fprop 16 e8k2 fp4 weights", "op": "moe_fprop", "tokens": 16, "k": 2,
         "experts": 8, "inn": 4096, "out": 11008, "scaling": "mx", "fa": "e4m3", "fb": "e2m1",
         "pad": 16},
        # the 7B up-projection's weight to 4 bits, both ways, and back
        {"name": "fp4_cast 11008x4096 both", "op": "fp4_cast", "rows": 11008, "cols": 4096,
         "both": True},
        # a few rows of activations to 4 bits and back: latency
        {"name": "fp4_cast 16x4096", "op": "fp4_cast", "rows": 16, "cols": 4096, "both": False},
        # one token through the 7B up-projection with 4-bit weights
        {"name": "fp4_gemm 1x11008x4096 e4m3", "op": "fp4_gemm", "M": 1, "N": 11008, "K": 4096,
         "fa": "e4m3"},
        # the GPT-175B MLP share with both sides in 4 bits (the largest)
        {"name": "fp4_gemm 4096x49152x12288", "op": "fp4_gemm", "M": 4096, "N": 49152,
         "K": 12288, "fa": "e2m1"},
    ]


def _size(rng, lo, hi, step):
    """A size spread over the logarithm of [lo, hi], an odd multiple of step."""
    n = int(math.exp(rng.uniform(math.log(lo), math.log(hi))))
    return step * max(1, (n // step) | 1)


def _any(rng, lo, hi, step):
    """The same, but odd half of the time."""
    return _size(rng, lo, hi, 1 if rng.random() < 0.5 else step)


def draw(rng):
    op = rng.choice(["rms_fwd", "rms_bwd", "moe_fprop", "moe_dgrad", "moe_wgrad", "fp4_cast",
                     "fp4_gemm"])
    if op.startswith("rms"):
        cols = _any(rng, 64, 16384, 128)
        rows = min(_any(rng, 1, 16384, 16), max(1, (1 << 26) // cols))
        c = {"op": op, "rows": rows, "cols": cols, "x": rng.choice(["bf16", "f32"]),
             "w": rng.choice(["bf16", "f32"]), "ckpt": rng.random() < 0.5}
        if op == "rms_bwd":
            c["dres"] = rng.random() < 0.7
            return c
        c["delta"] = rng.random() < 0.7
        c["yq"] = rng.choice(["none", "tensor", "block", "mx"])
        c["y"] = c["yq"] == "none" or rng.random() < 0.5
        return c
    if op.startswith("moe"):
        scaling = rng.choice(["tensor", "block", "mx"])
        step = {"tensor": 16, "block": 128, "mx": 32}[scaling]
        pad = 128 if scaling == "block" or (op == "moe_wgrad" and scaling == "mx") else 16
        experts = rng.choice([6, 8, 16, 40, 64, 128])
        c = {"op": op, "tokens": _any(rng, 1, 8192, 16), "k": rng.choice([1, 2, 4, 6]),
             "experts": experts, "scaling": scaling, "pad": pad,
             "inn": _size(rng, 128, 4096, step)}
        # weights of at most 2^28 elements
        most = max(128, min(11008, (1 << 28) // (experts * c["inn"])))
        c["out"] = _size(rng, 64, most, 128 if scaling == "block" else rng.choice([1, 16, 64]))
        c["fa"] = rng.choice(["e4m3", "e5m2"])
        c["fb"] = rng.choice(["e4m3", "e5m2"] if scaling != "mx" or op == "moe_wgrad"
                             else ["e4m3", "e5m2", "e2m1"])
        return c
    if op == "fp4_cast":
        both = rng.random() < 0.5
        cols = _size(rng, 64, 16384, 32)
        rows = min(_size(rng, 32, 16384, 32) if both else _any(rng, 1, 16384, 16),
                   max(1, (1 << 26) // cols // 32) * 32)
        return {"op": op, "rows": rows, "cols": cols, "both": both}
    c = {"op": op, "M": _any(rng, 1, 8192, 16), "N": _any(rng, 64, 16384, 64),
         "K": _size(rng, 128, 12288, rng.choice([32, 128, 128]))}
    c["fa"] = rng.choice(["e4m3", "e5m2", "e2m1"])
    return c


# ----------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _tiles(v, b):
    """[rows][cols] -> [rows][tiles][b], the last tile filled up with zeros."""
    r, c = v.shape
    n = -(-c // b)
    return torch.nn.functional.pad(v, (0, n * b - c)).reshape(r, n, b)


def _mx_exponent(amax, fmt):
    """The least e with amax <= fmax * 2^e; 0 for blocks of zeros."""
    m, x = torch.frexp(amax)
    # 448 = 0.875 * 2^9, 57344 = 0.875 * 2^16, 6 = 0.75 * 2^3
    top, p = {"e4m3": (0.875, 9), "e5m2": (0.875, 16), "e2m1": (0.75, 3)}[fmt]
    e = torch.where(m <= top, x - p, x - p + 1).clamp(-127, 127)
    return torch.where(amax == 0, torch.zeros_like(e), e)


def _e2m1_values(v):
    """v (|v| <= 6) rounded to the nearest E2M1 value, ties to the even code."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(v.dtype)
    return torch.copysign(torch.round(a / step) * step, v)


def _e2m1_codes(v):
    """The codes of E2M1 values, packed two a byte, the first in the low half."""
    grid = torch.tensor(E2M1, device=v.device)
    c = torch.bucketize(v.abs(), grid).to(torch.uint8) + 8 * torch.signbit(v).to(torch.uint8)
    return (c[:, 0::2] + 16 * c[:, 1::2]).contiguous()


def _quant(v, b, mx, fmt):
    """32-bit v with one scale per row and b columns: (scaled and clamped
    values, the factors that bring them back; for mx the exponents)."""
    r, c = v.shape
    t = _tiles(v, b)
    amax = t.abs().amax(2)
    if mx:
        e = _mx_exponent(amax, fmt)
        scale = torch.ldexp(torch.ones_like(amax), -e)
    else:
        scale = torch.where((amax > 0) & (amax <= FLT_MAX), (FMAX[fmt] / amax).clamp(max=FLT_MAX),
                            torch.ones_like(amax))
    q = (t * scale[:, :, None]).clamp(-FMAX[fmt], FMAX[fmt]).view(r, -1)[:, :c]
    return q, (e if mx else 1.0 / scale)


def _bytes(q, fmt):
    if fmt == "e2m1":
        return _e2m1_codes(_e2m1_values(q))
    return q.to(FP8[fmt][0]).contiguous().view(torch.uint8)


def _e8m0(e):
    return (e + 127).to(torch.uint8)


def _operand_of(v, scaling, fmt, square=False):
    """v as a quantised operand in hand: bytes [rows][cols] and scales.
    square: 128x128 blocks under the blockwise recipe."""
    if scaling == "tensor":
        s = FMAX[fmt] / v.abs().amax()
        return _bytes((v * s).clamp(-FMAX[fmt], FMAX[fmt]), fmt), (1.0 / s).view(1)
    if scaling == "mx":
        q, e = _quant(v, 32, True, fmt)
        return _bytes(q, fmt), _e8m0(e)
    if not square:
        q, s = _quant(v, 128, False, fmt)
        return _bytes(q, fmt), s
    r, c = v.shape
    t = v.view(r // 128, 128, c // 128, 128)
    s = FMAX[fmt] / t.abs().amax((1, 3)).clamp(min=1e-30)
    q = (t * s[:, None, :, None]).clamp(-FMAX[fmt], FMAX[fmt]).reshape(r, c)
    return _bytes(q, fmt), 1.0 / s


def _segments(g, case):
    """Segment starts of a batch's choices sorted by expert, as int32 on the
    device, and (row is a token's, rows in all)."""
    t, k, e, pad = case["tokens"], case["k"], case["experts"], case["pad"]
    load = 0.7 * _normal(g, e)
    noise = -torch.log(-torch.log(torch.rand((t, e), generator=g, device=DEV) * 0.9998 + 1e-4))
    expert = torch.topk(load + noise, k, dim=1)[1]
    counts = (expert.reshape(-1, 1) == torch.arange(e, device=DEV)).sum(0)
    ends = torch.cumsum((counts + pad - 1) // pad * pad, 0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    n = expert.numel()
    rows = (n + min(n, e) * (pad - 1)) // pad * pad
    at = torch.arange(rows, device=DEV)
    seg = torch.searchsorted(ends, at, right=True).clamp(max=e - 1)
    real = (at < ends[-1]) & (at - offsets[seg] < counts[seg])
    return offsets.int(), real, rows


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    empty = lambda dt, *shape: torch.empty(shape, dtype=dt, device=DEV)  # noqa: E731
    if op.startswith("moe"):
        e, inn, out = case["experts"], case["inn"], case["out"]
        s["offsets"], real, rows = _segments(g, case)
        s["rows"] = rows
        # padding rows hold zeros, as a dispatch leaves them
        a = _normal(g, rows, inn if op != "moe_wgrad" else out) * real[:, None]
        if op == "moe_wgrad":
            # the gradients' and the rows' copies with the tokens contiguous
            s["a"], s["a_s"] = _operand_of(a.t().contiguous(), case["scaling"], case["fa"])
            b = _normal(g, rows, inn) * real[:, None]
            s["b"], s["b_s"] = _operand_of(b.t().contiguous(), case["scaling"], case["fb"])
            s["c"] = empty(torch.bfloat16, e, out, inn)
            return s
        s["a"], s["a_s"] = _operand_of(a, case["scaling"], case["fa"])
        w = [_operand_of(_normal(g, out, inn) * inn ** -0.5, case["scaling"], case["fb"], True)
             for _ in range(e)]
        s["b"] = torch.stack([q for q, _ in w])
        s["b_s"] = torch.stack([f for _, f in w])
        # rows past the last segment are not part of the result: they stay zero
        s["c"] = torch.zeros((rows, out), dtype=torch.bfloat16, device=DEV)
        return s
    if op == "fp4_gemm":
        m, n, k = case["M"], case["N"], case["K"]
        s["a"], s["a_s"] = _operand_of(_normal(g, m, k), "mx", case["fa"])
        s["b"], s["b_s"] = _operand_of(_normal(g, n, k) * k ** -0.5, "mx", "e2m1")
        s["c"] = empty(torch.bfloat16, m, n)
        return s
    r, c = case["rows"], case["cols"]
    if op == "fp4_cast":
        # a weight's or an activation's columns have magnitudes of their own
        s["x_in"] = (_normal(g, r, c) * torch.exp(_normal(g, 1, c))).bfloat16()
        s["q"], s["q_s"] = empty(torch.uint8, r, c // 2), empty(torch.uint8, r, c // 32)
        s["y_out"] = empty(torch.bfloat16, r, c)
        if case["both"]:
            s["qT"], s["qT_s"] = empty(torch.uint8, c, r // 2), empty(torch.uint8, c, r // 32)
            s["yT_out"] = empty(torch.bfloat16, c, r)
        return s
    # rows of a residual stream: a few wide channels
    wide = torch.where(torch.rand(c, generator=g, device=DEV) < 0.01, 8.0, 1.0)
    x = (_normal(g, r, c) * wide).to(TYPES[case["x"]])
    s["gamma"] = (1.0 + 0.2 * _normal(g, c)).to(TYPES[case["w"]])
    s["rstd"] = empty(torch.float32, r)
    if op == "rms_fwd":
        s["x_in"] = x
        if case["delta"]:
            s["delta_in"] = (0.3 * _normal(g, r, c)).bfloat16()
            s["h"] = empty(TYPES[case["x"]], r, c)
        if case["y"]:
            s["y_out"] = empty(torch.bfloat16, r, c)
        if case["yq"] == "tensor":       # delayed scaling: the scale of the steps before
            s["q"] = empty(torch.uint8, r, c)
            s["scale"] = torch.full((1,), 32.0, dtype=torch.float32, device=DEV)
            s["amax"] = empty(torch.float32, 1)
        elif case["yq"] != "none":
            s["q"] = empty(torch.uint8, r, c)
            s["q_s"] = (empty(torch.float32, r, -(-c // 128)) if case["yq"] == "block"
                        else empty(torch.uint8, r, -(-c // 32)))
        if case["ckpt"]:
            s["ck"], s["ck_s"] = empty(torch.uint8, r, c), empty(torch.float32, r, -(-c // 128))
        return s
    x32 = x.float()
    s["rstd"] = 1.0 / torch.sqrt((x32 * x32).mean(1) + EPS)
    if case["ckpt"]:
        q, s["ck_s"] = _quant(x32 * s["rstd"][:, None], 128, False, "e4m3")
        s["ck"] = _bytes(q, "e4m3")
    else:
        s["x_in"] = x
    s["dy"] = (1e-3 * _normal(g, r, c)).bfloat16()
    if case["dres"]:
        s["dres_in"] = (1e-3 * _normal(g, r, c)).to(TYPES[case["x"]])
    s["dx"], s["dgamma"] = empty(TYPES[case["x"]], r, c), empty(torch.float32, c)
    return s


# -------------------------------------------------------------- plain form
def _unpack(q, fmt):
    """An operand's bytes as 32-bit values."""
    if fmt != "e2m1":
        return q.view(FP8[fmt][0]).float()
    v = torch.tensor(E2M1 + [-x for x in E2M1], device=q.device)
    pair = torch.stack([v.repeat(16), v.repeat_interleave(16)], 1)     # of each byte
    return pair[q.int()].view(*q.shape[:-1], 2 * q.shape[-1])


def _factors(f, scaling):
    return torch.ldexp(torch.ones((), device=f.device), f.int() - 127) if scaling == "mx" else f


def _spread(f, b, c):
    """Factors of b columns each over c columns."""
    return f.repeat_interleave(b, -1)[..., :c]


def _values(q, f, scaling, fmt, square=False):
    """What a quantised operand [..., rows][cols] stands for, in 32 bits."""
    v = _unpack(q, fmt)
    f = _factors(f, scaling)
    if scaling == "tensor":
        return v * f.view(-1, *[1] * (v.dim() - 1)) if v.dim() == 3 else v * f
    f = _spread(f, 32 if scaling == "mx" else 128, v.shape[-1])
    return v * (f.repeat_interleave(128, -2) if square and scaling == "block" else f)


def _held(q, f):
    """An 8-bit checkpoint's values."""
    return q.view(torch.float8_e4m3fn).float() * _spread(f, 128, q.shape[1])


def _plain(s):
    op, out = s["op"], {}
    if op.startswith("moe"):
        # a program without grouped products reads the segments' sizes and
        # launches one product an expert
        a = _values(s["a"], s["a_s"], s["scaling"], s["fa"])
        at = s["offsets"].tolist()
        if op == "moe_wgrad":
            b = _values(s["b"], s["b_s"], s["scaling"], s["fb"])
            parts = [a[:, i:j] @ b[:, i:j].t() for i, j in zip(at, at[1:])]
            return {"dw": torch.stack(parts).bfloat16()}
        b = _values(s["b"], s["b_s"], s["scaling"], s["fb"], True)
        parts = [a[i:j] @ w.t() for w, i, j in zip(b, at, at[1:])]
        parts.append(a.new_zeros((s["rows"] - at[-1], s["out"])))
        return {"y": torch.cat(parts).bfloat16()}
    if op == "fp4_gemm":
        a = _values(s["a"], s["a_s"], "mx", s["fa"])
        return {"y": (a @ _values(s["b"], s["b_s"], "mx", "e2m1").t()).bfloat16()}
    if op == "fp4_cast":
        for way in ("", "T") if s["both"] else ("",):
            x = s["x_in"].float()
            q, e = _quant(x.t() if way else x, 32, True, "e2m1")
            f = torch.ldexp(torch.ones((), device=q.device), e)
            out["y" + way] = (_e2m1_values(q) * _spread(f, 32, q.shape[1])).bfloat16()
            out["scale" + way] = _e8m0(e).view(torch.float8_e8m0fnu)
        return out
    gamma = s["gamma"].float()
    if op == "rms_fwd":
        x = s["x_in"].float()
        if s["delta"]:
            out["h"] = (x + s["delta_in"].float()).to(TYPES[s["x"]])
            x = out["h"].float()
        rstd = 1.0 / torch.sqrt((x * x).mean(1) + EPS)
        xhat = x * rstd[:, None]
        y = xhat * gamma
        out["rstd"] = rstd
        if s["y"]:
            out["y"] = y.bfloat16()
        if s["yq"] == "tensor":
            out["q"] = (y * 32.0).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            out["amax"] = y.abs().amax().view(1)
        elif s["yq"] != "none":
            mx = s["yq"] == "mx"
            q, f = _quant(y, 32 if mx else 128, mx, "e4m3")
            out["q"] = q.to(torch.float8_e4m3fn)
            out["q_scale"] = _e8m0(f).view(torch.float8_e8m0fnu) if mx else f
        if s["ckpt"]:
            q, out["ck_scale"] = _quant(xhat, 128, False, "e4m3")
            out["ck"] = q.to(torch.float8_e4m3fn)
        return out
    rstd = s["rstd"][:, None]
    xhat = _held(s["ck"], s["ck_s"]) if s["ckpt"] else s["x_in"].float() * rstd
    dy = s["dy"].float()
    g = dy * gamma
    dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if s["dres"]:
        dx = dx + s["dres_in"].float()
    return {"dx": dx.to(TYPES[s["x"]]), "dgamma": (dy * xhat).sum(0)}


# -------------------------------------------------------- the framework's
def _framework(s):
    from scaled_fp8_gemm_amd import fp8sg as F
    op = s["op"]
    fmt = {"e4m3": F.E4M3, "e5m2": F.E5M2, "e2m1": F.FP4_E2M1}
    if op.startswith("moe"):
        row = {"tensor": F.SCALE_TENSOR, "block": F.SCALE_BLOCK_1x128, "mx": F.SCALE_MX_1x32}
        a = F.operand(s["a"], fmt[s["fa"]], row[s["scaling"]], s["a_s"])
        if op == "moe_wgrad":
            b = F.operand(s["b"], fmt[s["fb"]], row[s["scaling"]], s["b_s"])
            F.fp8_gemm_grouped_wgrad(a, b, s["offsets"], s["experts"], s["rows"], s["out"],
                                     s["inn"], s["c"])
            return {"dw": s["c"]}
        if "w" not in s:         # weights keep their operand
            s["w"] = F.operand(s["b"], fmt[s["fb"]], F.SCALE_BLOCK_128x128
                               if s["scaling"] == "block" else row[s["scaling"]], s["b_s"])
        if op == "moe_fprop":
            F.fp8_gemm_grouped_fprop(a, s["w"], s["offsets"], s["experts"], s["rows"], s["out"],
                                     s["inn"], s["c"])
        else:
            F.fp8_gemm_grouped_dgrad(a, s["w"], s["offsets"], s["experts"], s["rows"], s["inn"],
                                     s["out"], s["c"])
        return {"y": s["c"]}
    if op == "fp4_gemm":
        if "w" not in s:
            s["w"] = F.operand(s["b"], F.FP4_E2M1, F.SCALE_MX_1x32, s["b_s"])
        F.fp8_gemm_fprop(F.operand(s["a"], fmt[s["fa"]], F.SCALE_MX_1x32, s["a_s"]), s["w"],
                         s["M"], s["N"], s["K"], s["c"])
        return {"y": s["c"]}
    if op == "fp4_cast":
        r, c = s["rows"], s["cols"]
        if s["both"]:
            F.fp8_quantize_mx4_t(s["x_in"], s["q"], s["q_s"], s["qT"], s["qT_s"])
        else:
            F.fp8_quantize_mx4(s["x_in"], s["q"], s["q_s"])
        F.fp8_dequantize_mx4(s["q"], s["q_s"], r, c, s["y_out"])
        out = {"y": s["y_out"], "scale": s["q_s"].view(torch.float8_e8m0fnu)}
        if s["both"]:
            F.fp8_dequantize_mx4(s["qT"], s["qT_s"], c, r, s["yT_out"])
            out.update(yT=s["yT_out"], scaleT=s["qT_s"].view(torch.float8_e8m0fnu))
        return out
    if op == "rms_fwd":
        yq = ck = None
        if s["yq"] != "none":
            scaling = {"tensor": F.SCALE_TENSOR, "block": F.SCALE_BLOCK_1x128,
                       "mx": F.SCALE_MX_1x32}[s["yq"]]
            yq = F.cast_out(s["q"], F.E4M3, scaling, s.get("q_s"), s.get("scale"), s.get("amax"))
        if s["yq"] == "tensor" and "ws" not in s:
            s["ws"] = F.workspace()
        if s["ckpt"]:
            ck = F.cast_out(s["ck"], F.E4M3, F.SCALE_BLOCK_1x128, s["ck_s"])
        F.fp8_rmsnorm_fwd(s["x_in"], s.get("delta_in"), s["gamma"], EPS, s.get("h"),
                          s.get("y_out"), s["rstd"], yq=yq, xhat=ck, workspace=s.get("ws"))
        out = {"rstd": s["rstd"]}
        if s["delta"]:
            out["h"] = s["h"]
        if s["y"]:
            out["y"] = s["y_out"]
        if yq is not None:
            out["q"] = s["q"].view(torch.float8_e4m3fn)
            if s["yq"] == "tensor":
                out["amax"] = s["amax"]
            else:
                out["q_scale"] = (s["q_s"].view(torch.float8_e8m0fnu) if s["yq"] == "mx"
                                  else s["q_s"])
        if s["ckpt"]:
            out["ck"], out["ck_scale"] = s["ck"].view(torch.float8_e4m3fn), s["ck_s"]
        return out
    if "ws" not in s:
        s["ws"] = F.rmsnorm_workspace(s["rows"], s["cols"])
    ck = F.operand(s["ck"], F.E4M3, F.SCALE_BLOCK_1x128, s["ck_s"]) if s["ckpt"] else None
    F.fp8_rmsnorm_bwd(s["dy"], s.get("x_in"), s["rstd"], s["gamma"], s.get("dres_in"), s["dx"],
                      s["dgamma"], xhat=ck, workspace=s["ws"])
    return {"dx": s["dx"], "dgamma": s["dgamma"]}


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------- in 64 bits
def _exact_operand(q, f, scaling, fmt, square=False):
    """The operand's values, decoded from the formats' bit fields."""
    b = q.long()
    if fmt == "e2m1":
        b = torch.stack([b % 16, b // 16], -1).view(*q.shape[:-1], -1)
        bits, bias, sign = 1, 1, 8
    else:
        bits, bias, sign = (3, 7, 128) if fmt == "e4m3" else (2, 15, 128)
    m, e = b % (1 << bits), b % sign // (1 << bits)
    v = torch.where(e == 0, m.double() * 2.0 ** (1 - bias - bits),
                    (1 + m.double() / (1 << bits)) * torch.exp2(e.double() - bias))
    v = torch.where(b >= sign, -v, v)
    f = torch.exp2(f.double() - 127) if scaling == "mx" else f.double()
    if scaling == "tensor":
        return v * (f.view(-1, 1, 1) if v.dim() == 3 else f)
    f = f.repeat_interleave(32 if scaling == "mx" else 128, -1)[..., :v.shape[-1]]
    if square and scaling == "block":
        f = f.repeat_interleave(128, -2)
    return v * f


def _exact_mx4(x):
    """(values of the nearest E2M1 codes, E8M0 factors) of x's blocks of 32."""
    r, c = x.shape
    t = x.view(r, c // 32, 32)
    big = t.abs().amax(2)
    f = torch.exp2(torch.ceil(torch.log2(big / 6)))
    # log2 may land an ulp off at a power of two: settle it by comparing
    f = torch.where(big > 6 * f, 2 * f, f)
    f = torch.where(big <= 3 * f, f / 2, f)
    f = torch.where(big == 0, torch.ones_like(f), f)
    a, code = t.abs() / f[:, :, None], torch.zeros_like(t)
    for i in range(7):           # past the middle between codes i and i + 1?
        mid = (E2M1[i] + E2M1[i + 1]) / 2
        code += (a > mid) | ((a == mid) & (i % 2 == 1))
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    v = torch.where(t < 0, -1.0, 1.0) * grid[code.long()] * f[:, :, None]
    return v.view(r, c), f


def _exact_cast(v, b, mx):
    """(v / factor, factor) without rounding: the values that the bytes and
    scales of an E4M3 cast with b-column blocks approximate."""
    r, c = v.shape
    n = -(-c // b)
    big = v.new_zeros((r, n * b))
    big[:, :c] = v.abs()
    big = big.view(r, n, b).amax(2)
    if mx:
        factor = torch.exp2(torch.ceil(torch.log2(big / 448)))
        factor = torch.where(big > 448 * factor, 2 * factor, factor)
        factor = torch.where(big <= 224 * factor, factor / 2, factor)
    else:
        factor = big / 448
    factor = torch.where(big == 0, torch.ones_like(big), factor)
    return v / factor.repeat_interleave(b, 1)[:, :c], factor


def exact(case, seed):
    s = prepare(case, seed)
    op, out = case["op"], {}
    if op.startswith("moe"):
        a = _exact_operand(s["a"], s["a_s"], case["scaling"], case["fa"])
        at = s["offsets"].tolist()
        c = torch.zeros(s["c"].shape, dtype=torch.float64, device=DEV)
        for e in range(case["experts"]):
            i, j = at[e], at[e + 1]
            if op == "moe_wgrad":
                if e == 0:
                    b = _exact_operand(s["b"], s["b_s"], case["scaling"], case["fb"])
                c[e] = a[:, i:j] @ b[:, i:j].t()
            else:
                w = _exact_operand(s["b"][e], s["b_s"][e], case["scaling"], case["fb"], True)
                c[i:j] = a[i:j] @ w.t()
        return {"dw" if op == "moe_wgrad" else "y": c}
    if op == "fp4_gemm":
        a = _exact_operand(s["a"], s["a_s"], "mx", case["fa"])
        return {"y": a @ _exact_operand(s["b"], s["b_s"], "mx", "e2m1").t()}
    if op == "fp4_cast":
        x = s["x_in"].double()
        out["y"], out["scale"] = _exact_mx4(x)
        if case["both"]:
            out["yT"], out["scaleT"] = _exact_mx4(x.t().contiguous())
        return out
    gamma = s["gamma"].double()
    if op == "rms_fwd":
        x = s["x_in"].double()
        if case["delta"]:
            out["h"] = x + s["delta_in"].double()
            # the norm is that of the stream as it is stored
            x = out["h"].float().to(TYPES[case["x"]]).double()
        out["rstd"] = (x.square().mean(1) + EPS).rsqrt()
        xhat = x * out["rstd"][:, None]
        y = xhat * gamma
        if case["y"]:
            out["y"] = y
        if case["yq"] == "tensor":
            out["q"], out["amax"] = (32 * y).clamp(-448, 448), y.abs().max().view(1)
        elif case["yq"] != "none":
            mx = case["yq"] == "mx"
            out["q"], out["q_scale"] = _exact_cast(y, 32 if mx else 128, mx)
        if case["ckpt"]:
            out["ck"], out["ck_scale"] = _exact_cast(xhat, 128, False)
        return out
    rstd, dy = s["rstd"].double()[:, None], s["dy"].double()
    xhat = (_exact_operand(s["ck"], s["ck_s"], "block", "e4m3") if case["ckpt"]
            else s["x_in"].double() * rstd)
    g, n = dy * gamma, case["cols"]
    out["dx"] = rstd / n * (n * g - xhat * (g * xhat).sum(1, True))
    if case["dres"]:
        out["dx"] = out["dx"] + s["dres_in"].double()
    out["dgamma"] = (dy * xhat).sum(0)
    return out


# -------------------------------------------------------------------- work
def _operand_bytes(scaling, fmt, r, c):
    """Bytes of an operand [r][c] with its scales."""
    data = r * c // 2 if fmt == "e2m1" else r * c
    return data + {"tensor": 4, "block": 4 * r * -(-c // 128), "mx": r * -(-c // 32),
                   "square": r * c // 4096}[scaling]


def work(case):
    op = case["op"]
    if op.startswith("moe"):
        n, e, inn, out = case["tokens"] * case["k"], case["experts"], case["inn"], case["out"]
        sc, fa, fb = case["scaling"], case["fa"], case["fb"]
        if op == "moe_wgrad":
            read = _operand_bytes(sc, fa, n, out) + _operand_bytes(sc, fb, n, inn)
            return {"bytes": read + 2 * e * out * inn, "flops": 2 * n * inn * out}
        used = min(e, n)         # experts that can have a token
        read = _operand_bytes(sc, fa, n, inn) + used * _operand_bytes(
            "square" if sc == "block" else sc, fb, out, inn)
        return {"bytes": read + 2 * n * out, "flops": 2 * n * inn * out}
    if op == "fp4_gemm":
        m, n, k = case["M"], case["N"], case["K"]
        return {"bytes": _operand_bytes("mx", case["fa"], m, k) + _operand_bytes("mx", "e2m1", n, k)
                + 2 * m * n, "flops": 2 * m * n * k}
    r, c = case["rows"], case["cols"]
    n = r * c
    if op == "fp4_cast":
        ways = 2 if case["both"] else 1
        return {"bytes": 2 * n + ways * (2 * _operand_bytes("mx", "e2m1", r, c) + 2 * n),
                "flops": 3 * n * ways}
    xb, wb = {"bf16": 2, "f32": 4}[case["x"]], {"bf16": 2, "f32": 4}[case["w"]]
    held = _operand_bytes("block", "e4m3", r, c) if case["ckpt"] else 0
    if op == "rms_fwd":
        q = 0 if case["yq"] == "none" else _operand_bytes(case["yq"], "e4m3", r, c)
        return {"bytes": xb * n + ((2 + xb) * n if case["delta"] else 0) + (2 * n if case["y"] else 0)
                + q + held + 4 * r + wb * c, "flops": 6 * n}
    return {"bytes": 2 * n + (held or xb * n) + (xb * n if case["dres"] else 0) + xb * n + 4 * r
            + wb * c + 4 * c, "flops": 11 * n}
