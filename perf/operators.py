"""The microscaled operators of the compressed linear layer, as cases to measure.

    W ~= S + U V^T + D     S: CSR outliers, U V^T: low rank, D: 4-bit microscaled (MXFP4)

kinds of a case
    "apply"   Y = X (S + U V^T + D)^T, bf16: serving, from one token to a prefill
    "dgrad"   dX = G (S + U V^T + D), bf16: the input gradient, with the same stored D
    "fp4"     a weight to MXFP4 and back, with the residual W - D that a factorisation takes next
    "int8"    an activation to its 8-bit checkpoint (MXINT8) and back
    "wgrad"   dS (on S's support), dU, dV^T in fp32 from the 8-bit checkpoint of X and the upstream gradient

`own` false: plain torch; true: the library's calls.  Both read the same stored arrays.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 32  # columns that share one scale


def _case(name, kind, m, n, b=0, r=0, frac=0.0, dtype="bf16"):
    return {"name": name, "kind": kind, "m": m, "n": n, "b": b, "r": r, "frac": frac, "dtype": dtype}


def listed():
    return [
        # one token through an attention projection whose outliers are kept apart: launch latency counts
        _case("apply_4096x4096_b1", "apply", 4096, 4096, b=1, frac=0.005),
        # one token through an MLP projection with a rank-64 correction: the stream of the 4-bit weights counts
        _case("apply_11008x4096_b1", "apply", 11008, 4096, b=1, r=64),
        # a handful of sequences decoded together, nothing a multiple of anything
        _case("apply_2731x5003_b13", "apply", 2731, 5003, b=13, r=37, frac=0.01),
        # a prefill of 2048 tokens: matrix cores
        _case("apply_8192x8192_b2048", "apply", 8192, 8192, b=2048, r=64, frac=0.005),
        # fine-tuning S, U, V over a frozen D: the input gradient of a down projection
        _case("dgrad_4096x11008_b2048", "dgrad", 4096, 11008, b=2048, r=64, frac=0.005),
        # the same for a short ragged batch without a low-rank term
        _case("dgrad_2049x1999_b77", "dgrad", 2049, 1999, b=77, frac=0.01),
        # compressing one MLP projection held in fp32
        _case("fp4_4096x11008_f32", "fp4", 4096, 11008, dtype="f32"),
        # and an odd bf16 one
        _case("fp4_1001x4099_bf16", "fp4", 1001, 4099),
        # the checkpoint of 2048 tokens at the input of a down projection
        _case("int8_2048x11008", "int8", 2048, 11008),
        # the smallest checkpoint: one token
        _case("int8_1x4096", "int8", 1, 4096),
        # parameter gradients of a large layer over a full batch
        _case("wgrad_8192x8192_b2048", "wgrad", 8192, 8192, b=2048, r=128, frac=0.03),
        # and of an odd one over a few tokens
        _case("wgrad_1501x2777_b201", "wgrad", 1501, 2777, b=201, r=41, frac=0.02),
    ]


def _log(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(["apply", "apply", "dgrad", "fp4", "int8", "wgrad"])
    m, n = _log(rng, 64, 11008), _log(rng, 64, 11008)
    while m * n > 8192 * 8192:
        m, n = _log(rng, 64, 11008), _log(rng, 64, 11008)
    if kind == "fp4":
        return {"kind": kind, "m": m, "n": n, "b": 0, "r": 0, "frac": 0.0, "dtype": rng.choice(["f32", "bf16"])}
    if kind == "int8":
        return {"kind": kind, "m": _log(rng, 1, 2048), "n": n, "b": 0, "r": 0, "frac": 0.0, "dtype": "bf16"}
    b = _log(rng, 1, 2048)
    r = rng.choice([0, rng.randint(1, 128), 8 * rng.randint(1, 16)])
    frac = rng.choice([0.0, round(rng.uniform(0.001, 0.03), 4)])
    if kind == "wgrad":
        r, frac = max(r, 1), max(frac, 0.001)
    return {"kind": kind, "m": m, "n": n, "b": b, "r": r, "frac": frac, "dtype": "bf16"}


def work(case):
    m, n, b, r = case["m"], case["n"], case["b"], case["r"]
    el = 4 if case["dtype"] == "f32" else 2
    nnz = case["frac"] * m * n
    if case["kind"] == "fp4":  # W in; the values (bf16) and the residual out
        return {"bytes": m * n * (el + 2 + el), "flops": 4.0 * m * n}
    if case["kind"] == "int8":
        return {"bytes": m * n * (el + 2), "flops": 3.0 * m * n}
    if case["kind"] == "wgrad":  # the checkpoint, G, the factors and S's pattern in; the fp32 gradients out
        return {"bytes": b * n * (1 + 1 / 32) + 2.0 * b * m + 4 * nnz + 2.0 * r * (m + n) + 4 * nnz + 4.0 * r * (m + n),
                "flops": 2.0 * b * nnz + 4.0 * b * r * (m + n)}
    return {"bytes": m * n * (0.5 + 1 / 32) + 6 * nnz + 2.0 * r * (m + n) + 2.0 * b * (m + n),
            "flops": 2.0 * b * m * n + 2.0 * b * r * (m + n)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed, stream):
    return torch.Generator(device=DEV).manual_seed(1000003 * seed + stream)


def _weight(m, n, seed):
    """A heavy-tailed weight (Student t, 3 degrees of freedom), as trained projections have."""
    g = _gen(seed, 1)
    den = torch.randn(m, n, device=DEV, generator=g).square_()
    den += torch.randn(m, n, device=DEV, generator=g).square_()
    den += torch.randn(m, n, device=DEV, generator=g).square_()
    return torch.randn(m, n, device=DEV, generator=g).mul_(0.02) / den.div_(3).sqrt_().clamp_(min=1e-3)


def _activation(b, n, seed, stream, scale):
    """Activations with a few loud channels."""
    g = _gen(seed, stream)
    loud = 1 + 15 * (torch.rand(n, device=DEV, generator=g) < 0.005).float()
    return (torch.randn(b, n, device=DEV, generator=g) * loud * scale).bfloat16()


def _inputs(case, seed):
    m, n, b, r = case["m"], case["n"], case["b"], case["r"]
    s = dict(case)
    if case["kind"] == "fp4":
        s["W"] = _weight(m, n, seed) if case["dtype"] == "f32" else _weight(m, n, seed).bfloat16()
        return s
    if case["kind"] == "int8":
        s["X"] = _activation(m, n, seed, 2, 1.0)
        return s
    W = _weight(m, n, seed).bfloat16().float()
    keep = W.abs().flatten().topk(int(case["frac"] * m * n), sorted=False).indices  # S: the largest weights, D: the rest
    mask = torch.zeros(m * n, dtype=torch.bool, device=DEV).index_fill_(0, keep, True).view(m, n)
    rows, cols = mask.nonzero(as_tuple=True)
    s["row_ptr"] = torch.zeros(m + 1, dtype=torch.int32, device=DEV)
    s["row_ptr"][1:] = mask.sum(1).cumsum(0).int()
    s["col_idx"], s["values"] = cols.int(), W[rows, cols].bfloat16()
    g = _gen(seed, 4)
    s["U"] = (0.05 * torch.randn(m, r, device=DEV, generator=g)).bfloat16()
    s["Vt"] = (0.05 * torch.randn(r, n, device=DEV, generator=g)).bfloat16()
    if case["kind"] == "wgrad":
        s["codes"], s["scales"] = _encode(_activation(b, n, seed, 5, 1.0).float(), "int8")
        s["G"] = _activation(b, m, seed, 6, 0.01)
        return s
    s["codes"], s["scales"] = _encode(W.masked_fill_(mask, 0), "fp4")
    if case["kind"] == "dgrad":
        s["G"] = _activation(b, m, seed, 6, 0.01)
    else:
        s["X"] = _activation(b, n, seed, 5, 1.0)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # the handles and buffers that a program keeps
        import sparse_rank_linear_hss_amd as hss
        s["hss"] = hss
        if case["kind"] == "fp4":
            s["q"] = hss.MXTensor.empty("fp4", case["m"], case["n"], DEV)
            s["D"] = torch.empty(case["m"], case["n"], dtype=torch.bfloat16, device=DEV)
            s["R"] = torch.empty_like(s["W"])
        elif case["kind"] == "int8":
            s["q"] = hss.MXTensor.empty("int8", case["m"], case["n"], DEV)
            s["D"] = torch.empty(case["m"], case["n"], dtype=torch.bfloat16, device=DEV)
        else:
            mx = None
            if case["kind"] != "wgrad":
                mx = hss.MXTensor("fp4", case["m"], case["n"], s["codes"], s["scales"])
            A = hss.HSSMatrix("csr", case["m"], case["n"], torch.bfloat16, U=s["U"], Vt=s["Vt"],
                              row_ptr=s["row_ptr"], col_idx=s["col_idx"], values=s["values"], mx=mx)
            if case["kind"] == "wgrad":
                s["A"], s["ckpt"] = A, hss.MXTensor("int8", case["b"], case["n"], s["codes"], s["scales"])
                s["ws"] = hss.grad_ckpt_workspace(A, case["b"], DEV)
                s["out"] = {"dS": torch.empty(A.nnz, device=DEV), "dU": torch.empty(case["m"], case["r"], device=DEV),
                            "dVt": torch.empty(case["r"], case["n"], device=DEV)}
            else:
                s["A"] = A if case["kind"] == "apply" else hss.hss_transposed_layer(A)
                s["ws"] = s["A"].workspace(case["b"], DEV)
                s["Y"] = torch.empty(case["b"], s["A"].m, dtype=torch.bfloat16, device=DEV)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    hss = s["hss"]
    if s["kind"] == "fp4":
        hss.hss_mx_quantize(s["W"], "fp4", out=s["q"], residual=s["R"])
        return {"values": hss.hss_mx_dequantize(s["q"], out=s["D"]), "residual": s["R"]}
    if s["kind"] == "int8":
        hss.hss_mx_quantize(s["X"], "int8", out=s["q"])
        return {"values": hss.hss_mx_dequantize(s["q"], out=s["D"])}
    if s["kind"] == "wgrad":
        return hss.hss_grad_ckpt(s["A"], s["ckpt"], s["G"], out=s["out"], ws=s["ws"])
    return hss.hss_apply(s["A"], s["X"] if s["kind"] == "apply" else s["G"], s["Y"], s["ws"])


def _plain(s):
    if s["kind"] == "fp4":
        W = s["W"].float()
        D = _decode(*_encode(W, "fp4"), W.shape[1], "fp4")
        return {"values": D.bfloat16(), "residual": (W - D).to(s["W"].dtype)}
    if s["kind"] == "int8":
        X = s["X"].float()
        return {"values": _decode(*_encode(X, "int8"), X.shape[1], "int8").bfloat16()}
    U, Vt = s["U"].float(), s["Vt"].float()
    rows = torch.repeat_interleave(torch.arange(s["m"], device=DEV), s["row_ptr"].diff())
    at = (rows, s["col_idx"].long())
    if s["kind"] == "wgrad":
        X, G = _decode(s["codes"], s["scales"], s["n"], "int8"), s["G"].float()
        return {"dS": (G.T @ X)[at], "dU": G.T @ (X @ Vt.T), "dVt": (G @ U).T @ X}
    W = _decode(s["codes"], s["scales"], s["n"], "fp4")
    W[at] += s["values"].float()
    if s["kind"] == "apply":
        X = s["X"].float()
        return (X @ W.T + (X @ Vt.T) @ U.T).bfloat16()
    G = s["G"].float()
    return (G @ W + (G @ U) @ Vt).bfloat16()


def _pow2(e):
    """2^e exactly, e whole and within a normal fp32's range."""
    return ((e + 127) << 23).view(torch.float32)


def _encode(w, fmt):
    """Groups of 32 columns: the exponent of the largest magnitude, rounded to the code's precision first (2 bits of
    an E2M1 value, 7 of an 8-bit integer), gives the shared power of two; then each value to the nearest code."""
    rows, cols = w.shape
    groups = -(-cols // GROUP)
    w = torch.nn.functional.pad(w, (0, groups * GROUP - cols)).view(rows, groups, GROUP)
    bits, top = (2, 2) if fmt == "fp4" else (7, 6)
    mant, ex = torch.frexp(w.abs().amax(2))
    e = ex - 1 + (torch.round(mant * 2 ** bits) == 2 ** bits).int()
    e = e.clamp(-123, 127) if fmt == "fp4" else e.clamp(-120, 127)
    v = w * _pow2(top - e)[..., None]
    if fmt == "int8":
        return v.round().clamp(-127, 127).to(torch.int8).view(rows, -1), (e + 127).to(torch.uint8)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = ((a / step).round() * step).clamp(max=6)
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) | (v.signbit().to(torch.uint8) << 3)
    return (code[..., 0::2] | code[..., 1::2] << 4).view(rows, -1), (e - 2 + 127).to(torch.uint8)


def _decode(codes, scales, cols, fmt):
    rows, groups = scales.shape
    if fmt == "int8":
        v = codes.view(rows, groups, GROUP) * _pow2(scales.int() - 133)[..., None]
    else:
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
        code = torch.stack([codes & 15, codes >> 4], 2).view(rows, groups, GROUP)
        v = grid[code.int()] * _pow2(scales.int() - 127)[..., None]
    return v.view(rows, -1)[:, :cols]


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    if case["kind"] in ("fp4", "int8"):
        src = s["W"] if case["kind"] == "fp4" else s["X"]
        near = _nearest64(src.double(), case["kind"])
        if case["kind"] == "int8":
            return {"values": near}
        return {"values": near, "residual": src.double() - near}
    m, n = case["m"], case["n"]
    S = torch.zeros(m * n, dtype=torch.float64, device=DEV)
    count = s["row_ptr"].long()
    owner = torch.searchsorted(count, torch.arange(len(s["col_idx"]), device=DEV), right=True) - 1
    place = owner * n + s["col_idx"].long()
    S[place] = s["values"].double()
    U, V = s["U"].double(), s["Vt"].double().T
    if case["kind"] == "wgrad":
        X = (s["codes"] * _two64(s["scales"].int().repeat_interleave(GROUP, 1) - 133))[:, :n]
        G = s["G"].double()
        return {"dS": torch.matmul(G.T, X).flatten()[place], "dU": torch.matmul(G.T, torch.matmul(X, V)),
                "dVt": torch.matmul(torch.matmul(X.T, G), U).T}
    # E2M1 by its fields: sign, two exponent bits, one mantissa bit
    q = torch.empty(m, s["codes"].shape[1] * 2, dtype=torch.int32, device=DEV)
    q[:, 0::2], q[:, 1::2] = (s["codes"] % 16).int(), (s["codes"] // 16).int()
    ex, frac = (q // 2) % 4, (q % 2).double()
    D = torch.where(ex == 0, 0.5 * frac, (1 + 0.5 * frac) * _two64(ex - 1)) * (1 - 2 * (q // 8))
    D = (D * _two64(s["scales"].int().repeat_interleave(GROUP, 1) - 127))[:, :n]
    A = torch.matmul(U, V.T) + D + S.view(m, n)
    return torch.matmul(s["X"].double(), A.T) if case["kind"] == "apply" else torch.matmul(s["G"].double(), A)


def _two64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest64(w, fmt):
    rows, cols = w.shape
    groups = -(-cols // GROUP)
    a = torch.zeros(rows, groups * GROUP, dtype=torch.float64, device=DEV)
    a[:, :cols] = w.abs()
    a = a.view(rows, groups, GROUP)
    largest = a.max(2).values
    e = torch.frexp(largest).exponent - 1
    # the largest magnitude rounds up to the next power of two from here on
    carry = largest >= (2 - (0.25 if fmt == "fp4" else 2.0 ** -7)) * _two64(e)
    e = torch.clamp(e + carry.int(), -123 if fmt == "fp4" else -120, 127)
    if fmt == "int8":
        step = _two64(e - 6)[..., None]
        near = torch.clamp(torch.floor(a / step + 0.5), max=127)
        near = near - ((near - a / step == 0.5) & (near % 2 == 1)).double()  # a tie goes to the even integer
    else:
        step = _two64(e - 2)[..., None]
        v = a / step  # halfway values go to the code whose last bit is 0
        index = (v > 0.25).int() + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5)
        near = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)[index]
    return (near * step).view(rows, -1)[:, :cols] * torch.sign(w)
