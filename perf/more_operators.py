"""Adapters beside the compressed layer and the optimizer of its factors, as cases to measure.

kinds of a case
    "apply"   Y = base + the rows' own adapters: row t of Y gains scale_l (x_t Vt_l^T) U_l^T, l = ids[t] (none: no
              adapter), bf16; base is the shared projection's output.  From one token to a prefill, many requests at once
    "grad"    the same layer's backward pass: dX = base + scale_l (g_t U_l) Vt_l in bf16 (base: the shared projection's
              part), dU_l = scale_l G_l^T (X_l Vt_l^T) and dVt_l = scale_l (G_l U_l)^T X_l in fp32 for every adapter
    "adamw"   one AdamW step over the trained tensors of a decoder layer (values of S, U, Vt of each projection): the
              moments in fp32, or in 8 bits, e4m3 times one fp32 scale for each 256 elements

8-bit moments: m and sqrt(v) are divided by their block's scale (largest magnitude / 448) and rounded up or down at
random, in proportion, so that a slow average does not stop between two codes; a value of sqrt(v) above 0 takes the
smallest code at least.  The random number of an element is a hash of its position (blocks of 256 counted through the
tensors) and the step.  A block whose scale would fall below 2^-100 is kept as zeros.

`own` false: plain torch; true: the library's calls.  Both read the same stored arrays.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 256  # elements of a tensor that share one scale of the 8-bit moments
LR, BETA1, BETA2, EPS, DECAY = 1e-4, 0.9, 0.999, 1e-8, 0.01


def _adapters(name, kind, m, n, b, r, count, mix, bare=0.0):
    """count: adapters of the bank; mix: "rows" (a decode batch, each row its own request) or "runs" (requests of many
    rows, one behind the other); bare: the share of rows without an adapter."""
    return {"name": name, "kind": kind, "m": m, "n": n, "b": b, "r": r, "count": count, "mix": mix, "bare": bare}


def _adamw(name, hidden, inner, projections, r, frac, bits, p, g):
    """The first `projections` of q, k, v, o (hidden x hidden), gate, up (inner x hidden), down (hidden x inner); S holds
    `frac` of a weight.  p: "f32", "bf16", or "bf16+f32" (a master copy beside bf16 parameters); g: the gradients' type."""
    return {"name": name, "kind": "adamw", "hidden": hidden, "inner": inner, "projections": projections, "r": r,
            "frac": frac, "bits": bits, "p": p, "g": g, "step": 1000}


def listed():
    return [
        # one request's next token through an attention projection with a small adapter: launch latency counts
        _adapters("apply_4096x4096_b1_r16", "apply", 4096, 4096, 1, 16, 1, "rows"),
        # 64 requests decoded together, each with its own adapter: the stream of the adapters counts
        _adapters("apply_11008x4096_b64_r64_of64", "apply", 11008, 4096, 64, 64, 64, "rows"),
        # some requests with an adapter and some without, nothing a multiple of anything
        _adapters("apply_2731x5003_b77_r37_of9", "apply", 2731, 5003, 77, 37, 9, "rows", 0.2),
        # a prefill of 2048 tokens of four adapters at a down projection
        _adapters("apply_4096x11008_b2048_r64_of4", "apply", 4096, 11008, 2048, 64, 4, "runs"),
        # fine-tuning one small adapter of an attention projection over a full batch
        _adapters("grad_4096x4096_b2048_r16", "grad", 4096, 4096, 2048, 16, 1, "runs"),
        # eight adapters trained side by side at a gate projection
        _adapters("grad_11008x4096_b2048_r64_of8", "grad", 11008, 4096, 2048, 64, 8, "runs"),
        # the same for an odd layer and a ragged batch, part of it without an adapter
        _adapters("grad_1501x2777_b201_r41_of5", "grad", 1501, 2777, 201, 41, 5, "runs", 0.15),
        # a short sequence through a small layer
        _adapters("grad_1024x1024_b16_r8", "grad", 1024, 1024, 16, 8, 1, "runs"),
        # every factor of a decoder layer, mixed precision
        _adamw("adamw_layer_r409_bits32", 4096, 11008, 7, 409, 0.03, 32, "bf16+f32", "f32"),
        # the same with 8-bit moments
        _adamw("adamw_layer_r409_bits8", 4096, 11008, 7, 409, 0.03, 8, "bf16+f32", "f32"),
        # an odd layer in fp32 throughout
        _adamw("adamw_odd_r37_bits32", 1501, 2777, 7, 37, 0.01, 32, "f32", "f32"),
        # the factors of one small adapter, 8-bit moments, everything else in bf16: launch latency counts
        _adamw("adamw_adapter_r8_bits8", 1024, 1024, 1, 8, 0.0, 8, "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(["apply", "apply", "grad", "grad", "adamw", "adamw"])
    if kind == "adamw":
        while True:
            case = _adamw("", _log(rng, 64, 4096), _log(rng, 64, 11008), rng.randint(1, 7), _log(rng, 1, 409),
                          rng.choice([0.0, round(rng.uniform(0.001, 0.05), 4)]), rng.choice([8, 32]),
                          rng.choice(["f32", "bf16", "bf16+f32"]), rng.choice(["f32", "bf16"]))
            case["step"] = _log(rng, 1, 100000)
            if sum(_tensors(case)) <= 38_000_000:
                break
    else:
        while True:
            m, n, b, r, count = _log(rng, 64, 11008), _log(rng, 64, 11008), _log(rng, 1, 2048), _log(rng, 1, 128), _log(rng, 1, 64)
            if b * r * (m + n) <= 2048 * 64 * 15104 and count * r * (m + n) <= (64 if kind == "apply" else 8) * 64 * 15104:
                break
        case = _adapters("", kind, m, n, b, r, count, rng.choice(["rows", "runs"]), rng.choice([0.0, round(rng.uniform(0, 0.5), 2)]))
    del case["name"]
    return case


def _tensors(case):
    """The element counts of a step's tensors: S's values, U and Vt of each projection."""
    h, i = case["hidden"], case["inner"]
    sizes = []
    for m, n in [(h, h), (h, h), (h, h), (h, h), (i, h), (i, h), (h, i)][:case["projections"]]:
        sizes += [k for k in (int(case["frac"] * m * n), m * case["r"], n * case["r"]) if k > 0]
    return sizes


def work(case):
    if case["kind"] == "adamw":
        count = sum(_tensors(case))
        # what holds the parameter is read and written (its bf16 copy is written); so is each moment
        weight = {"f32": 8, "bf16": 4, "bf16+f32": 10}[case["p"]]
        state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        return {"bytes": count * (weight + state + (4 if case["g"] == "f32" else 2)), "flops": 16.0 * count}
    m, n, b, r = case["m"], case["n"], case["b"], case["r"]
    live = min(case["count"], b)
    if case["kind"] == "apply":
        return {"bytes": 2.0 * b * (n + 2 * m) + 2.0 * live * r * (m + n), "flops": 2.0 * b * r * (m + n)}
    return {"bytes": 2.0 * b * (m + 3 * n) + 2.0 * live * r * (m + n) + 4.0 * case["count"] * r * (m + n),
            "flops": 2.0 * b * r * (2 * m + 3 * n)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed, stream):
    return torch.Generator(device=DEV).manual_seed(1000003 * seed + stream)


def _activation(b, n, seed, stream, scale):
    """Activations with a few loud channels."""
    g = _gen(seed, stream)
    loud = 1 + 15 * (torch.rand(n, device=DEV, generator=g) < 0.005).float()
    return (torch.randn(b, n, device=DEV, generator=g) * loud * scale).bfloat16()


def _inputs(case, seed):
    return _adamw_inputs(case, seed) if case["kind"] == "adamw" else _adapter_inputs(case, seed)


def _adapter_inputs(case, seed):
    m, n, b, r, count = case["m"], case["n"], case["b"], case["r"], case["count"]
    s = dict(case)
    g = _gen(seed, 1)
    s["U"] = (0.05 * torch.randn(count, m, r, device=DEV, generator=g)).bfloat16()
    s["Vt"] = (0.05 * torch.randn(count, r, n, device=DEV, generator=g)).bfloat16()
    s["scale"] = 0.25 + 1.75 * torch.rand(count, device=DEV, generator=g)
    who = torch.randperm(count, device=DEV, generator=g)
    if case["mix"] == "rows":  # a decode batch: the bank's adapters in turn, the rows in no order
        request = torch.randperm(b, device=DEV, generator=g)
    else:  # as many requests as adapters, of ragged lengths
        cuts = (torch.rand(min(count, b) - 1, device=DEV, generator=g) * b).long().sort().values
        request = torch.searchsorted(cuts, torch.arange(b, device=DEV), right=True)
    ids = who[request % count]
    s["ids"] = torch.where(torch.rand(b, device=DEV, generator=g) < case["bare"], -1, ids).int()
    s["X"] = _activation(b, n, seed, 2, 1.0)
    if case["kind"] == "apply":
        s["base"] = _activation(b, m, seed, 3, 1.0)
    else:
        s["G"], s["base"] = _activation(b, m, seed, 3, 0.01), _activation(b, n, seed, 4, 0.01)
    return s


def _adamw_inputs(case, seed):
    """One flat buffer for each kind of array; a tensor starts at a multiple of BLOCK elements, zeros between them."""
    s = dict(case)
    sizes = _tensors(case)
    s["sizes"], s["starts"], at = sizes, [], 0
    for k in sizes:
        s["starts"].append(at)
        at += -(-k // BLOCK) * BLOCK
    live = torch.zeros(at, dtype=torch.bool, device=DEV)
    for a, k in zip(s["starts"], sizes):
        live[a:a + k] = True
    g = _gen(seed, 5)

    def normal(scale):
        return torch.randn(at, device=DEV, generator=g) * live * scale

    # the size of a gradient differs from row to row of a factor, and so do its averages
    loud = torch.exp(1.5 * torch.randn(at // BLOCK, device=DEV, generator=g)).repeat_interleave(BLOCK) * 1e-3
    s["grad"] = (normal(1.0) * loud).to(torch.float32 if case["g"] == "f32" else torch.bfloat16)
    p = normal(0.05)
    if case["p"] == "f32":
        s["param"] = p
    else:
        s["param"] = p.bfloat16()
        if case["p"] == "bf16+f32":
            s["master"] = p
    m, root = normal(0.3) * loud, (1e-3 + torch.rand(at, device=DEV, generator=g)) * live * loud
    if case["bits"] == 32:
        s["m"], s["v"] = m, root * root
        return s
    for name, x in (("m", m), ("v", root)):
        scale = x.view(-1, BLOCK).abs().amax(1) / 448
        s[name] = (x.view(-1, BLOCK) / scale.clamp(min=1e-30)[:, None]).to(torch.float8_e4m3fn).view(-1)
        s[name + "_scale"] = scale
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # the handles and buffers that a program keeps
        import sparse_rank_linear_hss_amd as hss
        s["hss"] = hss
        if case["kind"] == "adamw":
            def parts(flat, per=1):
                return [flat[a // per:a // per + -(-k // per)] for a, k in zip(s["starts"], s["sizes"])]
            kept = {k: parts(s[k]) for k in ("master", "m", "v") if k in s}
            kept |= {k: parts(s[k], BLOCK) for k in ("m_scale", "v_scale") if k in s}
            s["state"] = hss.AdamWState(parts(s["param"]), bits=case["bits"], **kept)
            s["grads"] = parts(s["grad"])
            return s
        s["bank"] = hss.HSSAdapters(s["U"], s["Vt"], s["scale"])
        if case["kind"] == "apply":
            s["ws"] = hss.adapters_workspace(s["bank"], case["b"], DEV)
            s["Y"] = torch.empty_like(s["base"])
        else:
            s["ws"] = hss.adapters_grad_workspace(s["bank"], case["b"], DEV)
            s["out"] = {"dX": torch.empty_like(s["base"]), "dU": torch.empty(s["U"].shape, device=DEV),
                        "dVt": torch.empty(s["Vt"].shape, device=DEV)}
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    hss = s["hss"]
    if s["kind"] == "apply":
        return hss.hss_adapters_apply(s["bank"], s["X"], s["ids"], base=s["base"], Y=s["Y"], ws=s["ws"])
    if s["kind"] == "grad":
        return hss.hss_adapters_grad(s["bank"], s["X"], s["G"], s["ids"], base=s["base"], out=s["out"], ws=s["ws"])
    hss.hss_adamw(s["state"], s["grads"], lr=LR, step=s["step"], betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY)
    return _updated(s)


def _updated(s):
    return {k: s[k] for k in ("param", "master", "m", "v", "m_scale", "v_scale") if k in s}


def _plain(s):
    if s["kind"] == "adamw":
        return _plain_adamw(s)
    U, Vt, X = s["U"].float(), s["Vt"].float(), s["X"].float()
    count, m, r = U.shape
    # every row times every adapter of the bank, kept where the adapter is the row's own
    mine = ((s["ids"][:, None] == torch.arange(count, device=DEV)) * s["scale"]).repeat_interleave(r, 1)
    Ur, Vr = U.transpose(1, 2).reshape(count * r, m), Vt.reshape(count * r, -1)
    T = (X @ Vr.T) * mine
    if s["kind"] == "apply":
        return (s["base"].float() + T @ Ur).bfloat16()
    G = s["G"].float()
    P = (G @ Ur.T) * mine
    return {"dX": (s["base"].float() + P @ Vr).bfloat16(), "dU": (T.T @ G).view(count, r, m).transpose(1, 2).contiguous(),
            "dVt": (P.T @ X).view(count, r, -1)}


def _plain_adamw(s):
    t = s["step"]
    weight = s["master"] if "master" in s else s["param"]
    g = s["grad"].float()
    m = BETA1 * _value(s, "m") + (1 - BETA1) * g
    root = _value(s, "v")
    v = BETA2 * (root * root if s["bits"] == 8 else root) + (1 - BETA2) * (g * g)
    root = torch.sqrt(v)
    denom = root * (1 / math.sqrt(1 - BETA2 ** t)) + EPS
    p = weight.float() * (1 - LR * DECAY) - (LR / (1 - BETA1 ** t)) * (m / denom)
    if weight is not s["param"]:
        weight.copy_(p)
    s["param"].copy_(p)
    if s["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        h = _hash(len(g), t)
        _keep(s, "m", m, h & 0xffff, 0)
        _keep(s, "v", root, (h >> 16) & 0xffff, 1)
    return _updated(s)


def _value(s, name):
    if s["bits"] == 32:
        return s[name]
    return (s[name].float().view(-1, BLOCK) * s[name + "_scale"][:, None]).view(-1)


def _wrap(x):
    """x mod 2^32 as a signed number of 32 bits."""
    x &= 0xffffffff
    return x - (1 << 32) if x >> 31 else x


def _hash(count, step):
    """32 bits for each position: multiplications by odd constants (the first digits of the golden ratio and of the
    square roots of 3, 2 and 19) modulo 2^32, with the upper bits folded onto the lower ones in between."""
    h = torch.arange(count, dtype=torch.int32, device=DEV) * _wrap(0x9E3779B1) + _wrap(step * 0xBB67AE85)
    h = (h ^ ((h >> 16) & 0xffff)) * _wrap(0x6A09E667)
    h = (h ^ ((h >> 15) & 0x1ffff)) * _wrap(0x5BE0CD19)
    return h ^ ((h >> 16) & 0xffff)


def _keep(s, name, x, u, least):
    """x in 8 bits: u / 2^16 of a step is added before the bits below the step are dropped."""
    x = x.view(-1, BLOCK)
    scale = x.abs().amax(1) * (1 / 448)
    scale = torch.where(scale < 2.0 ** -100, 0.0, scale)
    inv = torch.where(scale > 0, 1 / scale, 0.0)
    a = (x.abs() * inv[:, None]).clamp(max=448).view(-1)
    normal = ((a.view(torch.int32) + (u << 4)) >> 20) - 960
    small = (a * 512 + u * 2.0 ** -16).int()
    code = torch.where(a < 2.0 ** -6, small, normal).clamp(max=126)
    code = torch.where((x.view(-1) != 0) & (scale > 0).repeat_interleave(BLOCK), code.clamp(min=least), code)
    code = code | (x.view(-1).signbit().int() << 7)
    s[name].view(torch.uint8).copy_(code)
    s[name + "_scale"].copy_(scale)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    if case["kind"] == "adamw":
        return _exact_adamw(s)
    out = s["base"].double()
    dU = torch.zeros(s["U"].shape, dtype=torch.float64, device=DEV)
    dVt = torch.zeros(s["Vt"].shape, dtype=torch.float64, device=DEV)
    for k in range(case["count"]):
        rows = (s["ids"] == k).nonzero().view(-1)
        if not len(rows):
            continue
        U, V, scale = s["U"][k].double(), s["Vt"][k].double().T.contiguous(), s["scale"][k].double()
        X = s["X"][rows].double()
        T = torch.matmul(X, V)
        if case["kind"] == "apply":
            out[rows] += scale * torch.matmul(T, U.T)
            continue
        G = s["G"][rows].double()
        P = torch.matmul(G, U)
        out[rows] += scale * torch.matmul(P, V.T)
        dU[k] = scale * torch.matmul(G.T, T)
        dVt[k] = scale * torch.matmul(P.T, X)
    return out if case["kind"] == "apply" else {"dX": out, "dU": dU, "dVt": dVt}


def _exact_adamw(s):
    t, count = s["step"], len(s["grad"])
    g = s["grad"].double()
    if s["bits"] == 8:
        by = {k: s[k + "_scale"].double().repeat_interleave(BLOCK) for k in ("m", "v")}
        m, v = s["m"].double() * by["m"], (s["v"].double() * by["v"]) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = m + (1 - BETA1) * (g - m)
    v = v + (1 - BETA2) * (g ** 2 - v)
    w = s["master" if "master" in s else "param"].double()
    w = w - LR * DECAY * w - LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)) ** 0.5 + EPS)
    out = {"param": w, "m": m, "v": v}
    if "master" in s:
        out["master"] = w
    if s["bits"] == 8:
        random = _hash64(count, t)
        for name, x, u in (("m", m, random % 65536), ("v", v ** 0.5, random // 65536)):
            out[name + "_scale"] = x.view(-1, BLOCK).abs().max(1).values / 448
            per = out[name + "_scale"].repeat_interleave(BLOCK)
            a = torch.nan_to_num(x.abs() / per).clamp(max=448)
            # a step of e4m3: 2^-3 of the value's power of two, 2^-9 at the least
            step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
            a = torch.clamp(torch.floor(a / step + u.double() / 65536) * step, max=448)
            if name == "v":
                a = torch.where(x > 0, a.clamp(min=2.0 ** -9), a)
            out[name] = a * torch.sign(x)
    return out


def _hash64(count, step):
    mod = 1 << 32
    h = (torch.arange(count, dtype=torch.int64, device=DEV) * 0x9E3779B1 + (step * 0xBB67AE85) % mod) % mod
    for shift, factor in ((65536, 0x6A09E667), (32768, 0x5BE0CD19)):
        h = torch.bitwise_xor(h, h // shift)
        # the product in two halves of the factor: it would not fit 63 bits
        h = (h * (factor % 65536) + (h * (factor // 65536) % 65536) * 65536) % mod
    return torch.bitwise_xor(h, h // 65536)
