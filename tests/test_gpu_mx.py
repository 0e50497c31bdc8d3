"""GPU parity of the microscaled operators against the CPU oracle: quantisation
bit for bit, apply and gradients within derived bounds.

Bounds.  u = 2^-24 (half a step of fp32), bf16's half step 2^-8 relative.
A sum of K products in fp32, in any order, is off by at most K u times the sum
of magnitudes N (products of bf16 values are exact).  Apply: the fp32 sums
(X V: n terms, then n + 2 r), T in two bf16 terms (2^-16 of T), D + S rounded
to bf16 where they meet (2^-8 of the weight, only asked for where the test
makes them meet), then Y rounded (2^-8 of Y):
    |err| <= 2^-8 |Y| + ((2 n + 2 r + 2) u + 2^-16 + meet 2^-8) N.
Gradients, T and P in three bf16 terms (2^-24 of them, in u below):
    |err| <= (K + 3 b + 2) u N,  K = n (dU), m (dV), 0 (dS)."""
import numpy as np
import pytest

import hss_synth as syn
import oracle as O
from _cases import to_dev, to_host

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24
BF = O.BF16


@pytest.fixture(scope="module")
def H():
    import sparse_rank_linear_hss_amd as h
    return h


def _raw(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _tdt(dtype):
    import torch
    return torch.float32 if dtype == O.F32 else torch.bfloat16


# ---------------------------------------------------------------------------
# Quantisation
# ---------------------------------------------------------------------------

def _check_quantise(H, W, dtype, fmt, Wd=None):
    import torch
    W64 = O.widen(W, dtype)
    rows, cols = W64.shape
    codes, scales = O.mx_encode(W64, fmt)
    Wd = to_dev(W, dtype) if Wd is None else Wd
    q, res = H.hss_mx_quantize(Wd, fmt, residual=True)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    D = O.mx_decode(codes, scales, cols, fmt)
    for dt in (torch.float32, torch.bfloat16):
        got = H.hss_mx_dequantize(q, dt).float().cpu().numpy().astype(np.float64)
        assert np.array_equal(got, D, equal_nan=True)
    want = np.where(np.isnan(D), np.nan, np.where(np.isfinite(W64), W64, np.nan) - D)
    assert np.array_equal(res.float().cpu().numpy().astype(np.float64), want, equal_nan=True)
    H.hss_mx_quantize(Wd, fmt, out=q, residual=Wd)                  # the residual over W itself
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.array_equal(Wd.float().cpu().numpy(), res.float().cpu().numpy(), equal_nan=True)


@pytest.mark.parametrize("fmt", ["fp4", "int8"])
@pytest.mark.parametrize("dtype", [O.F32, BF])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (3, 32), (5, 33), (2, 64), (17, 95), (33, 131), (4, 1000), (700, 3)])
def test_quantise(H, fmt, dtype, shape):
    W = syn.random_matrix(*shape, dtype, seed=11 + shape[0] * 7 + shape[1], kind="t3")
    _check_quantise(H, W, dtype, fmt)


@pytest.mark.parametrize("fmt", ["fp4", "int8"])
@pytest.mark.parametrize("dtype", [O.F32, BF])
def test_quantise_edges(H, fmt, dtype):
    """Ties and carries at every code border, zeros of both signs, the type's
    largest and smallest values, and groups with NaN or infinities."""
    W = np.zeros((12, 64), np.float32)
    half = np.arange(32) / 4.0 if fmt == "fp4" else np.arange(32) * 4.0 + 0.5
    W[0, :32], W[0, 32:] = half, -half
    W[1, :32] = np.minimum(half, 6.75) if fmt == "fp4" else np.minimum(half, 127)
    W[2, ::2] = -0.0
    W[3] = np.float32(2.0 ** -126)
    W[4] = np.float32(2.0 ** -133)                                  # a denormal (also of bf16)
    W[5, 3] = np.array([0x7F7F0000], np.uint32).view(np.float32)[0]
    W[6, 3], W[6, 40] = np.nan, 1.0
    W[7, 33], W[7, 1] = -np.inf, 2.0
    W[8] = 2.0 ** np.linspace(-120, 120, 64)
    W[9, 0] = 7.0 if fmt == "fp4" else 127.5
    W[10, 0], W[10, 1] = -7.0, 3.5
    if dtype == BF:
        W = (W.view(np.uint32) >> 16).astype(np.uint16)
    _check_quantise(H, W, dtype, fmt)


def test_quantise_unaligned_source(H):
    """A source that starts 2 (bf16) or 4 (fp32) bytes past a 16-byte boundary."""
    import torch
    for dtype in (BF, O.F32):
        W = syn.random_matrix(9, 77, dtype, seed=3, kind="t3")
        buf = torch.zeros(9 * 77 + 1, dtype=_tdt(dtype), device="cuda")
        view = buf[1:].view(9, 77)
        view.copy_(to_dev(W, dtype))
        _check_quantise(H, W, dtype, "fp4", Wd=view)


# ---------------------------------------------------------------------------
# Apply
# ---------------------------------------------------------------------------

def _layer(H, m, n, r, seed, frac=(1, 100), col16=False, meet=False, empty_rows=False):
    """A layer W ~= S + U V^T + D: S the largest weights, D the rest in 4 bits
    (meet: D of the whole weight, so that S falls on non-zeros of D)."""
    import torch
    W = syn.random_matrix(m, n, BF, seed=seed, kind="t3")
    ref = O.split_csr(W, BF, O.topk_count(m, n, *frac))
    if empty_rows:
        ref = O.split_csr(np.where(np.arange(m)[:, None] % 3 == 0, W, np.uint16(0)), BF, min(m * n // 8, 40))
    S64 = O.dense_from_csr(m, n, ref["row_ptr"], ref["col_idx"], ref["values"], BF)
    W64 = O.widen(W, BF)
    codes, scales = O.mx_encode(W64 if meet else np.where(S64 != 0, 0, W64), "fp4")
    D64 = O.mx_decode(codes, scales, n, "fp4")
    k = len(ref["col_idx"])
    cols = ref["col_idx"].astype(np.uint16).view(np.int16) if col16 else ref["col_idx"]
    U, V = syn.factors(m, n, r, BF, seed) if r else (np.zeros((m, 0), np.uint16), np.zeros((n, 0), np.uint16))
    A = H.HSSMatrix("csr", m, n, torch.bfloat16, U=to_dev(U, BF) if r else None,
                    Vt=to_dev(np.ascontiguousarray(V.T), BF) if r else None,
                    row_ptr=_raw(ref["row_ptr"]) if k else None, col_idx=_raw(cols) if k else None,
                    values=to_dev(ref["values"], BF) if k else None, nnz=k,
                    mx=H.MXTensor("fp4", m, n, _raw(codes), _raw(scales)))
    return A, ref, S64, D64, O.widen(U, BF), O.widen(V, BF)


def _bounded(Y, S64, D64, U64, V64, X64, meet):
    """Y (device) against X (S + U V^T + D)^T."""
    n, r = X64.shape[1], U64.shape[1]
    Yref = X64 @ (S64 + D64).T + (X64 @ V64) @ U64.T
    N = np.abs(X64) @ (np.abs(S64) + np.abs(D64)).T + (np.abs(X64) @ np.abs(V64)) @ np.abs(U64).T
    bound = 2.0 ** -8 * np.abs(Yref) + ((2 * n + 2 * r + 2) * U24 + 2.0 ** -16 + (2.0 ** -8 if meet else 0)) * N
    err = np.abs(O.widen(to_host(Y), BF) - Yref)
    assert np.all(err <= bound), float(np.max(err / np.maximum(bound, 1e-300)))


APPLY = [
    # (m, n, r, b, options)
    (1, 1, 0, 1, {}), (5, 3, 1, 1, {}), (16, 32, 0, 1, {}), (64, 128, 8, 1, {}), (130, 96, 33, 3, {}),
    (257, 512, 0, 8, {}), (300, 1000, 41, 17, {}), (40, 38, 2, 2, {"meet": True}), (96, 4096, 64, 1, {}),
    (33, 4100, 5, 5, {"col16": True}), (129, 257, 7, 33, {"empty_rows": True}), (200, 300, 16, 64, {"col16": True}),
    (150, 640, 32, 65, {}), (256, 256, 64, 130, {"meet": True}), (131, 515, 9, 260, {}), (512, 1024, 128, 300, {}),
    (1030, 160, 24, 16, {}), (2100, 64, 3, 4, {}), (17, 12000, 0, 1, {}), (48, 8200, 40, 15, {}),
]


@pytest.mark.parametrize("trans", [False, True], ids=["fwd", "dgrad"])
@pytest.mark.parametrize("case", APPLY, ids=[f"{c[0]}x{c[1]}-r{c[2]}-b{c[3]}" for c in APPLY])
def test_apply(H, case, trans):
    m, n, r, b, opt = case
    A, ref, S64, D64, U64, V64 = _layer(H, m, n, r, seed=m * 3 + n, **opt)
    if trans:
        A = H.hss_transposed_layer(A)
        S64, D64, U64, V64 = S64.T, D64.T, V64, U64
    X = syn.random_matrix(b, A.n, BF, seed=b + 1, kind="normal", scale=1.0)
    Xd = to_dev(X, BF)
    Y = H.hss_apply(A, Xd)
    _bounded(Y, S64, D64, U64, V64, O.widen(X, BF), opt.get("meet", False))
    assert O.bits_equal(to_host(Y), to_host(H.hss_apply(A, Xd)))


@pytest.mark.parametrize("b", [1, 4, 17, 70])
@pytest.mark.parametrize("trans", [False, True], ids=["fwd", "dgrad"])
def test_apply_empty_parts(H, b, trans):
    """No S, no low-rank term: D alone; and a zero D (scale bytes of zeros' own)."""
    import torch
    m, n = 70, 129
    W = O.widen(syn.random_matrix(m, n, BF, seed=4, kind="t3"), BF)
    codes, scales = O.mx_encode(W, "fp4")
    mx = H.MXTensor("fp4", m, n, _raw(codes), _raw(scales))
    D64 = O.mx_decode(codes, scales, n, "fp4")
    A = H.HSSMatrix("csr", *((n, m) if trans else (m, n)), torch.bfloat16, mx=mx, mx_t=trans)
    X = syn.random_matrix(b, A.n, BF, seed=2, kind="normal", scale=1.0)
    zero = np.zeros((A.m, 0)), np.zeros((A.n, 0))
    D = D64.T if trans else D64
    _bounded(H.hss_apply(A, to_dev(X, BF)), np.zeros_like(D), D, *zero, O.widen(X, BF), False)
    z = H.hss_mx_quantize(torch.zeros(m, n, device="cuda"), "fp4")
    Z = H.HSSMatrix("csr", *((n, m) if trans else (m, n)), torch.bfloat16, mx=z, mx_t=trans)
    assert torch.count_nonzero(H.hss_apply(Z, to_dev(X, BF))) == 0


@pytest.mark.parametrize("b", [1, 12, 40, 300])
@pytest.mark.parametrize("trans", [False, True], ids=["fwd", "dgrad"])
def test_apply_non_finite(H, b, trans):
    """A non-finite group makes its outputs NaN and no other; a NaN in X its
    batch row, and no other."""
    import torch
    m, n = 96, 160
    W = O.widen(syn.random_matrix(m, n, BF, seed=9, kind="t3"), BF)
    W[37, 70] = np.inf
    codes, scales = O.mx_encode(W, "fp4")
    mx = H.MXTensor("fp4", m, n, _raw(codes), _raw(scales))
    A = H.HSSMatrix("csr", *((n, m) if trans else (m, n)), torch.bfloat16, mx=mx, mx_t=trans)
    X = to_dev(syn.random_matrix(b, A.n, BF, seed=2, kind="normal", scale=1.0), BF)
    hit = np.zeros(A.m, bool)
    hit[slice(64, 96) if trans else 37] = True
    Y = H.hss_apply(A, X).float().cpu().numpy()
    assert np.all(np.isnan(Y[:, hit])) and np.all(np.isfinite(Y[:, ~hit]))
    if b > 1:
        X[b - 1, 5] = float("nan")
        Y = H.hss_apply(A, X).float().cpu().numpy()
        assert np.all(np.isnan(Y[b - 1])) and np.all(np.isfinite(Y[:b - 1][:, ~hit]))


def test_apply_unaligned_operands_and_neighbours(H):
    """X, Y, U, Vt and values off the 16-byte grid, inside larger buffers whose
    other elements stay as they were."""
    import torch
    m, n, r = 67, 200, 24
    A, ref, S64, D64, U64, V64 = _layer(H, m, n, r, seed=77)

    def off(t):
        buf = torch.full((t.numel() + 9,), 7.0, dtype=t.dtype, device="cuda")
        buf[1:1 + t.numel()] = t.reshape(-1)
        return buf[1:1 + t.numel()].view(t.shape)

    B = H.HSSMatrix("csr", m, n, torch.bfloat16, U=off(A.U), Vt=off(A.Vt), row_ptr=A.row_ptr, col_idx=A.col_idx,
                    values=off(A.values), mx=A.mx)
    for b in (1, 7, 33, 150):
        X = syn.random_matrix(b, n, BF, seed=b, kind="normal", scale=1.0)
        out = torch.full((b * m + 18,), 7.0, dtype=torch.bfloat16, device="cuda")
        Y = out[9:9 + b * m].view(b, m)
        H.hss_apply(B, off(to_dev(X, BF)), Y)
        _bounded(Y, S64, D64, U64, V64, O.widen(X, BF), False)
        assert torch.all(out[:9] == 7) and torch.all(out[9 + b * m:] == 7)


def test_apply_group_noalloc_and_streams(H):
    """The grouped call, the call without a workspace and a call on another
    stream give the single call's bits."""
    import torch
    layers = [_layer(H, m, 256, r, seed=m) for m, r in ((100, 8), (64, 0), (33, 40))]
    for b in (1, 6, 40):
        X = to_dev(syn.random_matrix(b, 256, BF, seed=b, kind="normal", scale=1.0), BF)
        want = [to_host(H.hss_apply(l[0], X)) for l in layers]
        for w, y in zip(want, H.hss_apply_group([l[0] for l in layers], X)):
            assert O.bits_equal(w, to_host(y))
        for w, l in zip(want, layers):
            y = torch.empty((b, l[0].m), dtype=torch.bfloat16, device="cuda")
            assert O.bits_equal(w, to_host(H.hss_apply_noalloc(l[0], X, y)))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            ys = [H.hss_apply(l[0], X) for l in layers]
        s.synchronize()
        assert all(O.bits_equal(w, to_host(y)) for w, y in zip(want, ys))


# ---------------------------------------------------------------------------
# Gradients from an 8-bit checkpoint
# ---------------------------------------------------------------------------

def _check_grads(got, ref, N, n, m, b):
    K = {"dS": 0, "dU": n, "dV": m}
    for key, dev in (("dS", "dS"), ("dU", "dU"), ("dV", "dVt")):
        g = got[dev].cpu().numpy().astype(np.float64)
        g = g.T if key == "dV" else g
        bound = (K[key] + 3 * b + 2) * U24 * N[key]
        err = np.abs(g - ref[key])
        assert np.all(err <= bound), (key, float(np.max(err / np.maximum(bound, 1e-300))))


GRAD = [
    # (m, n, r, b, kind of S)
    (1, 1, 1, 1, "csr"), (7, 5, 2, 1, "csr"), (64, 96, 8, 33, "csr"), (130, 70, 33, 9, "col16"), (65, 260, 5, 64, "csr"),
    (40, 64, 12, 20, "2:4"), (128, 128, 64, 256, "csr"), (150, 200, 40, 520, "csr"), (96, 100, 16, 515, "2:4"),
    (300, 131, 130, 140, "csr"),
]


@pytest.mark.parametrize("route", ["auto", "sparse", "dense"])
@pytest.mark.parametrize("case", GRAD, ids=[f"{c[0]}x{c[1]}-r{c[2]}-b{c[3]}-{c[4]}" for c in GRAD])
def test_grad_ckpt(H, hss_opt, case, route):
    import torch
    m, n, r, b, kind = case
    hss_opt("grad_ds_route", route)
    if kind == "2:4":
        W = syn.random_matrix(m, n, BF, seed=m + n, kind="t3")
        s = O.split_24(W, BF)
        rp, ci = O.nm24_pattern(m, n, s["nm_meta"])
        U, V = syn.factors(m, n, r, BF, m)
        A = H.HSSMatrix("2:4", m, n, torch.bfloat16, U=to_dev(U, BF), Vt=to_dev(np.ascontiguousarray(V.T), BF),
                        nm_values=to_dev(s["nm_values"], BF), nm_meta=_raw(s["nm_meta"].view(np.int32)))
        U64, V64 = O.widen(U, BF), O.widen(V, BF)
    else:
        A, ref, _, _, U64, V64 = _layer(H, m, n, r, seed=m + n, frac=(5, 100), col16=kind == "col16")
        rp, ci = ref["row_ptr"], ref["col_idx"]
    X = syn.random_matrix(b, n, BF, seed=1, kind="normal", scale=1.0)
    G = syn.random_matrix(b, m, BF, seed=2, kind="normal", scale=0.01)
    ck = H.hss_mx_quantize(to_dev(X, BF), "int8")
    X64 = O.mx_decode(*O.mx_encode(O.widen(X, BF), "int8"), n, "int8")
    G64, S64 = O.widen(G, BF), np.zeros((m, n))
    ref_g = O.backward(m, n, rp, ci, S64, U64, V64, X64, G64)
    N = O.backward_normalisers(m, n, rp, ci, S64, U64, V64, X64, G64)
    got = H.hss_grad_ckpt(A, ck, to_dev(G, BF))
    _check_grads(got, ref_g, N, n, m, b)
    again = H.hss_grad_ckpt(A, ck, to_dev(G, BF))
    assert all(torch.equal(got[k], again[k]) for k in got)
    only = H.hss_grad_ckpt(A, ck, to_dev(G, BF), dS=False, dU=False)
    assert list(only) == ["dVt"] and torch.equal(only["dVt"], got["dVt"])
    only = H.hss_grad_ckpt(A, ck, to_dev(G, BF), dVt=False, dS=False)
    assert list(only) == ["dU"] and torch.equal(only["dU"], got["dU"])


def test_grad_ckpt_against_differences(H):
    """<gradient, direction> against the central difference of the loss
    L(S, U, V) = sum G o (X' (S + U V^T + D)^T) in fp64: L is quadratic along a
    direction, so the difference is exact but for rounding."""
    m, n, r, b = 48, 80, 6, 21
    A, ref, S64, D64, U64, V64 = _layer(H, m, n, r, seed=5)
    X = syn.random_matrix(b, n, BF, seed=1, kind="normal", scale=1.0)
    G = syn.random_matrix(b, m, BF, seed=2, kind="normal", scale=1.0)
    X64 = O.mx_decode(*O.mx_encode(O.widen(X, BF), "int8"), n, "int8")
    G64 = O.widen(G, BF)
    got = H.hss_grad_ckpt(A, H.hss_mx_quantize(to_dev(X, BF), "int8"), to_dev(G, BF))
    rng = np.random.default_rng(0)
    rows = O.csr_row_of_entry(m, ref["row_ptr"])
    dS = np.zeros((m, n))
    dS[rows, ref["col_idx"]] = rng.standard_normal(len(rows))
    dU, dV = rng.standard_normal((m, r)), rng.standard_normal((n, r))

    def loss(t):
        return float(np.sum(G64 * (X64 @ (S64 + t * dS + D64 + (U64 + t * dU) @ (V64 + t * dV).T).T)))

    diff = (loss(0.5) - loss(-0.5))
    inner = float(got["dS"].cpu().numpy().astype(float) @ dS[rows, ref["col_idx"]]
                  + np.sum(got["dU"].cpu().numpy() * dU) + np.sum(got["dVt"].cpu().numpy().T * dV))
    N = O.backward_normalisers(m, n, ref["row_ptr"], ref["col_idx"], S64, U64, V64, X64, G64)
    bound = sum(float(np.sum(N[k] * np.abs(d))) for k, d in (("dU", dU), ("dV", dV))) + float(
        np.sum(N["dS"] * np.abs(dS[rows, ref["col_idx"]])))
    assert abs(inner - diff) <= (max(m, n) + 3 * b + 2) * U24 * bound


def test_grad_ckpt_non_finite_token(H):
    """A token whose checkpoint group held a NaN reaches the gradients of that
    group's columns (dS, dV^T) and, through X' V, all of dU."""
    import torch
    m, n, r, b = 64, 96, 8, 40
    A, ref, *_ = _layer(H, m, n, r, seed=6)
    X = to_dev(syn.random_matrix(b, n, BF, seed=1, kind="normal", scale=1.0), BF)
    X[17, 40] = float("inf")
    G = to_dev(syn.random_matrix(b, m, BF, seed=2, kind="normal", scale=1.0), BF)
    got = H.hss_grad_ckpt(A, H.hss_mx_quantize(X, "int8"), G)
    hit = (np.asarray(ref["col_idx"]) >= 32) & (np.asarray(ref["col_idx"]) < 64)
    dS = got["dS"].cpu().numpy()
    assert np.all(np.isnan(dS[hit])) and np.all(np.isfinite(dS[~hit]))
    assert torch.isnan(got["dU"]).all() and torch.isnan(got["dVt"][:, 32:64]).all()
    assert torch.isfinite(got["dVt"][:, :32]).all() and torch.isfinite(got["dVt"][:, 64:]).all()


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

def test_training_step_over_a_frozen_dense_part(H):
    """split, quantise the rest, forward, checkpoint, backward (input and
    parameter gradients): each against the oracle's own chain."""
    import torch
    m, n, r, b = 200, 320, 16, 77
    W = syn.random_matrix(m, n, BF, seed=8, kind="t3")
    sp = H.hss_split(to_dev(W, BF), "csr", frac=(1, 100), residual=True)
    q, rest = H.hss_mx_quantize(sp.residual, "fp4", residual=True)
    U, V = syn.factors(m, n, r, BF, 3)
    A = H.HSSMatrix.from_split(sp, U=to_dev(U, BF), Vt=to_dev(np.ascontiguousarray(V.T), BF), mx=q)
    ref = O.split_csr(W, BF, sp.k)
    S64 = O.dense_from_csr(m, n, ref["row_ptr"], ref["col_idx"], ref["values"], BF)
    D64 = O.mx_decode(*O.mx_encode(O.widen(W, BF) - S64, "fp4"), n, "fp4")
    assert np.array_equal(rest.float().cpu().numpy(), O.widen(W, BF) - S64 - D64)   # what the factors are made from
    U64, V64 = O.widen(U, BF), O.widen(V, BF)
    X = syn.random_matrix(b, n, BF, seed=1, kind="normal", scale=1.0)
    G = syn.random_matrix(b, m, BF, seed=2, kind="normal", scale=0.01)
    Xd, Gd = to_dev(X, BF), to_dev(G, BF)
    _bounded(H.hss_apply(A, Xd), S64, D64, U64, V64, O.widen(X, BF), False)
    ck = H.hss_mx_quantize(Xd, "int8")
    g = H.hss_backward(A, ck, Gd)
    _bounded(g["dX"], S64.T, D64.T, V64, U64, O.widen(G, BF), False)
    X64 = O.mx_decode(*O.mx_encode(O.widen(X, BF), "int8"), n, "int8")
    args = (m, n, ref["row_ptr"], ref["col_idx"], S64, U64, V64, X64, O.widen(G, BF))
    _check_grads(g, O.backward(*args), O.backward_normalisers(*args), n, m, b)
    # with the input kept in bf16 instead, the same layer gives hss_grad's gradients
    full = H.hss_backward(A, Xd, Gd)
    assert torch.equal(full["dX"], g["dX"])


@pytest.mark.parametrize("b", [1, 9, 48, 200])
def test_captured_step_replays(H, b):
    """Forward, checkpoint, input gradient and parameter gradients in one
    graph, replayed with new inputs, other eager work in between."""
    import torch
    m, n, r = 160, 224, 24
    A, *_ = _layer(H, m, n, r, seed=12)
    At = H.hss_transposed_layer(A)
    X = torch.zeros(b, n, dtype=torch.bfloat16, device="cuda")
    G = torch.zeros(b, m, dtype=torch.bfloat16, device="cuda")
    Y, dX = torch.empty_like(G), torch.empty_like(X)
    ck = H.MXTensor.empty("int8", b, n, "cuda")
    out = {"dS": torch.empty(A.nnz, device="cuda"), "dU": torch.empty(m, r, device="cuda"),
           "dVt": torch.empty(r, n, device="cuda")}
    ws = [H.apply_workspace(H.hss_apply_workspace_size(L, b), "cuda") for L in (A, At)]
    gws = H.grad_ckpt_workspace(A, b, "cuda")

    def step():
        H.hss_apply(A, X, Y, ws[0])
        H.hss_mx_quantize(X, "int8", out=ck)
        H.hss_apply(At, G, dX, ws[1])
        H.hss_grad_ckpt(A, ck, G, out=out, ws=gws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(3):
        X.copy_(to_dev(syn.random_matrix(b, n, BF, seed=rep, kind="normal", scale=1.0), BF))
        G.copy_(to_dev(syn.random_matrix(b, m, BF, seed=rep + 9, kind="normal", scale=1.0), BF))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (Y, dX, out["dS"], out["dU"], out["dVt"])]
        e = [H.hss_apply(A, X), H.hss_apply(At, G)]
        g = H.hss_grad_ckpt(A, H.hss_mx_quantize(X, "int8"), G)
        want = e + [g["dS"], g["dU"], g["dVt"]]
        assert all(torch.equal(a, w) for a, w in zip(got, want))


def test_workspace_sized_for_the_largest_batch(H):
    """One workspace, of the size of the largest batch, for every smaller one:
    the bits of calls with workspaces of their own."""
    A = _layer(H, 400, 1536, 40, seed=31)[0]
    At = H.hss_transposed_layer(A)
    for L in (A, At):
        for top in (65, 129, 600):
            ws = H.apply_workspace(H.hss_apply_workspace_size(L, top), "cuda")
            for b in (1, 16, 17, 64, 65, 128, 129, 256, 257, 385, 559, 600):
                if b <= top:
                    X = to_dev(syn.random_matrix(b, L.n, BF, seed=b, kind="normal", scale=1.0), BF)
                    assert O.bits_equal(to_host(H.hss_apply(L, X, ws=ws)), to_host(H.hss_apply(L, X)))


def test_gradient_workspace_sized_for_the_largest_batch(H, hss_opt):
    """One workspace, of the size of the largest batch, for smaller ones and on
    either route of dS: the bits of calls with workspaces of their own."""
    import torch
    A = _layer(H, 700, 1300, 33, seed=32, frac=(3, 100))[0]
    ws = H.grad_ckpt_workspace(A, 1409, "cuda")
    for route in ("auto", "sparse", "dense"):
        hss_opt("grad_ds_route", route)
        for b in (1, 64, 257, 513, 1281, 1408, 1409):
            ck = H.hss_mx_quantize(to_dev(syn.random_matrix(b, A.n, BF, seed=b, kind="normal", scale=1.0), BF), "int8")
            G = to_dev(syn.random_matrix(b, A.m, BF, seed=b + 1, kind="normal", scale=1.0), BF)
            got, want = H.hss_grad_ckpt(A, ck, G, ws=ws), H.hss_grad_ckpt(A, ck, G)
            assert all(torch.equal(got[k], want[k]) for k in want), (route, b)


@pytest.mark.parametrize("kind", ["mx", "csr", "col16", "2:4", "empty"])
def test_transposed_layer_written_again(H, kind):
    """After S's values, U and V changed in place, the transposed layer written
    again holds the bits of a new one, in its old arrays; captured too."""
    import torch
    m, n, r = 96, 160, 12
    if kind == "2:4":
        W = to_dev(syn.random_matrix(m, n, BF, seed=2, kind="t3"), BF)
        U, V = syn.factors(m, n, r, BF, 2)
        A = H.HSSMatrix.from_split(H.hss_split(W, "2:4"), U=to_dev(U, BF), Vt=to_dev(np.ascontiguousarray(V.T), BF))
    else:
        A = _layer(H, m, n, 0 if kind == "empty" else r, seed=2, col16=kind == "col16",
                   frac=(0, 1) if kind == "empty" else (2, 100))[0]
        if kind == "csr":
            A = H.HSSMatrix("csr", m, n, torch.bfloat16, U=A.U, Vt=A.Vt, row_ptr=A.row_ptr, col_idx=A.col_idx,
                            values=A.values)
    At = H.hss_transposed_layer(A)
    held = [t for t in (At.values, At.U, At.Vt) if t is not None]
    where = [t.data_ptr() for t in held]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        H.hss_transposed_layer(A, out=At)
    for rep in range(4):
        for t in (A.values, A.nm_values, A.U, A.Vt):
            if t is not None:
                t.copy_(torch.randn(t.shape, device="cuda"))
        if rep % 2:
            graph.replay()
        else:
            assert H.hss_transposed_layer(A, out=At) is At
        new = H.hss_transposed_layer(A)
        torch.cuda.synchronize()
        for a, b in ((At.values, new.values), (At.U, new.U), (At.Vt, new.Vt)):
            assert (a is None and b is None) or torch.equal(a.view(torch.int16), b.view(torch.int16))
        G = torch.randn(9, m, device="cuda").bfloat16()
        assert torch.equal(H.hss_apply(At, G), H.hss_apply(new, G))
    assert where == [t.data_ptr() for t in held]


@pytest.mark.parametrize("route", ["sparse", "dense"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_grad_ckpt_non_finite_gradient(H, hss_opt, route, value):
    """A non-finite G[c][i] makes row i of dS and of dU, and all of dV^T,
    non-finite, and nothing else."""
    import torch
    hss_opt("grad_ds_route", route)
    m, n, r, b = 64, 96, 8, 70
    A, ref, *_ = _layer(H, m, n, r, seed=6, frac=(10, 100))
    X = torch.randn(b, n, device="cuda").bfloat16() + 3
    G = torch.randn(b, m, device="cuda").bfloat16()
    G[17, 40] = value
    got = H.hss_grad_ckpt(A, H.hss_mx_quantize(X, "int8"), G)
    hit = torch.arange(m, device="cuda") == 40
    rows = torch.as_tensor(O.csr_row_of_entry(m, ref["row_ptr"]), device="cuda")
    for name, at in (("dU", hit), ("dS", hit[rows])):
        assert not torch.isfinite(got[name][at]).any() and torch.isfinite(got[name][~at]).all()
    assert not torch.isfinite(got["dVt"]).any()
