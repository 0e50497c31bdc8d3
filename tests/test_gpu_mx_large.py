"""HSS_MX4 layers and checkpoint gradients at sizes that reach every large-tile
route: 256 x 256 and 256 x 192 tiles, K in one piece and split, with and
without a low-rank term, ragged edges, entries of S written from the tiles.

The plain implementation is torch in float64 on the GPU (decoding by field,
dense S, matmul); bounds as in test_gpu_mx.py, u = 2^-24."""
import pytest

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24


@pytest.fixture(scope="module")
def H():
    import sparse_rank_linear_hss_amd as h
    return h


def _layer(H, m, n, r, seed, density, col16=False):
    """Random codes, scales 2^-9 .. 2^-6, S at random places (D kept zero there)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    ng = -(-n // 32)
    codes = torch.randint(0, 256, (m, 16 * ng), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(118, 122, (m, ng), dtype=torch.uint8, device="cuda", generator=g)
    mask = torch.rand(m, n, device="cuda", generator=g) < density
    q = torch.empty(m, 32 * ng, dtype=torch.uint8, device="cuda")
    q[:, 0::2], q[:, 1::2] = codes & 15, codes >> 4
    q[:, n:] = 0
    q[:, :n][mask] = 0
    codes = (q[:, 0::2] | q[:, 1::2] << 4).contiguous()
    ex, frac = ((q >> 1) & 3).double(), (q & 1).double()
    val = torch.where(ex == 0, 0.5 * frac, (1 + 0.5 * frac) * 2.0 ** (ex - 1)) * (1 - 2 * (q >> 3).double())
    W = (val * 2.0 ** (scales.double() - 127).repeat_interleave(32, 1))[:, :n].contiguous()
    rows, cols = mask.nonzero(as_tuple=True)
    values = (0.1 * torch.randn(len(rows), device="cuda", generator=g)).bfloat16()
    W[rows, cols] += values.double()
    rp = torch.zeros(m + 1, dtype=torch.int32, device="cuda")
    rp[1:] = mask.sum(1).cumsum(0).int()
    U = (0.05 * torch.randn(m, r, device="cuda", generator=g)).bfloat16() if r else None
    Vt = (0.05 * torch.randn(r, n, device="cuda", generator=g)).bfloat16() if r else None
    A = H.HSSMatrix("csr", m, n, torch.bfloat16, U=U, Vt=Vt, row_ptr=rp, col_idx=cols.int() if len(cols) else None,
                    values=values if len(cols) else None, nnz=len(cols), mx=H.MXTensor("fp4", m, n, codes, scales))
    return (A.with_col16() if col16 else A), W, rows, cols


APPLY = [
    # (m, n, r, b, density)
    (4099, 700, 37, 2047, 0.01),     # 256 x 256 tiles, ragged on every side
    (11000, 640, 24, 2048, 0.0),     # 256 x 192 tiles
    (11000, 640, 0, 2041, 0.002),
    (513, 4200, 33, 385, 0.01),      # K split, 256 x 192 tiles
    (512, 4096, 0, 512, 0.0),
    (8192, 8192, 64, 1024, 0.001),   # K split, 256 x 256 tiles
    (2001, 1030, 300, 257, 0.005),   # the first batch past the middle route
    (900, 3001, 64, 256, 0.03),      # the last one of it
    (130, 9000, 8, 200, 0.001),
]


@pytest.mark.parametrize("trans", [False, True], ids=["fwd", "dgrad"])
@pytest.mark.parametrize("case", APPLY, ids=[f"{c[0]}x{c[1]}-r{c[2]}-b{c[3]}" for c in APPLY])
def test_apply_large(H, case, trans):
    import torch
    m, n, r, b, density = case
    A, W, _, _ = _layer(H, m, n, r, m + n + b, density, col16=b % 2 == 1)
    U, V = (A.U.double(), A.Vt.double().t()) if r else (None, None)
    if trans:
        A, W, U, V = H.hss_transposed_layer(A), W.t(), V, U
    g = torch.Generator(device="cuda").manual_seed(b)
    X = torch.randn(b, A.n, device="cuda", generator=g).bfloat16()
    out = torch.full((b * A.m + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = out[8:8 + b * A.m].view(b, A.m)
    H.hss_apply(A, X, Y)
    assert torch.all(out[:8] == 7) and torch.all(out[8 + b * A.m:] == 7)
    X64 = X.double()
    ref, N = X64 @ W.t().contiguous(), X64.abs() @ W.abs().t().contiguous()
    if r:
        Ut = U.t().contiguous()
        ref += (X64 @ V.contiguous()) @ Ut
        N += (X64.abs() @ V.abs().contiguous()) @ Ut.abs()
    bound = 2.0 ** -8 * ref.abs() + ((2 * A.n + 2 * r + 2) * U24 + 2.0 ** -16) * N
    err = (Y.double() - ref).abs()
    assert torch.all(err <= bound), float((err / bound.clamp(min=1e-300)).max())
    again = H.hss_apply(A, X)
    assert torch.equal(again, Y)


GRAD = [
    # (m, n, r, b, density)
    (3000, 2600, 130, 2048, 0.02), (700, 901, 12, 1500, 0.05), (257, 513, 64, 2047, 0.3), (4096, 1024, 16, 600, 0.001),
    (64, 11008, 40, 1025, 0.01),
]


@pytest.mark.parametrize("route", ["auto", "sparse", "dense"])
@pytest.mark.parametrize("case", GRAD, ids=[f"{c[0]}x{c[1]}-r{c[2]}-b{c[3]}" for c in GRAD])
def test_grad_ckpt_large(H, hss_opt, case, route):
    import torch
    m, n, r, b, density = case
    hss_opt("grad_ds_route", route)
    A, _, rows, cols = _layer(H, m, n, r, m + n, density, col16=b % 2 == 1)
    g = torch.Generator(device="cuda").manual_seed(b)
    X = torch.randn(b, n, device="cuda", generator=g)
    G = (0.01 * torch.randn(b, m, device="cuda", generator=g)).bfloat16()
    ck = H.hss_mx_quantize(X, "int8")
    X64, G64, U, Vt = H.hss_mx_dequantize(ck, torch.float32).double(), G.double(), A.U.double(), A.Vt.double()
    got = H.hss_grad_ckpt(A, ck, G)
    Gt, aGt, Vc = G64.t().contiguous(), G64.abs().t().contiguous(), Vt.t().contiguous()
    ref = {"dS": (Gt @ X64)[rows, cols], "dU": Gt @ (X64 @ Vc), "dVt": (G64 @ U).t().contiguous() @ X64}
    N = {"dS": (aGt @ X64.abs())[rows, cols], "dU": aGt @ (X64.abs() @ Vc.abs()),
         "dVt": (G64.abs() @ U.abs()).t().contiguous() @ X64.abs()}
    for key, K in (("dS", 0), ("dU", n), ("dVt", m)):
        err, bound = (got[key].double() - ref[key]).abs(), (K + 3 * b + 2) * U24 * N[key]
        assert torch.all(err <= bound), (key, float((err / bound.clamp(min=1e-300)).max()))
    again = H.hss_grad_ckpt(A, ck, G)
    assert all(torch.equal(got[k], again[k]) for k in got)


def test_grad_ckpt_2of4_large(H, hss_opt):
    """The tiles' output for a 2:4 pattern with a ragged last tile."""
    import torch
    hss_opt("grad_ds_route", "dense")
    m, n, r, b = 600, 1000, 16, 1100
    g = torch.Generator(device="cuda").manual_seed(3)
    W = torch.randn(m, n, device="cuda", generator=g).bfloat16()
    sp = H.hss_split(W, "2:4")
    U = (0.05 * torch.randn(m, r, device="cuda", generator=g)).bfloat16()
    Vt = (0.05 * torch.randn(r, n, device="cuda", generator=g)).bfloat16()
    A = H.HSSMatrix.from_split(sp, U=U, Vt=Vt)
    _, cols = H.hss_nm24_to_csr(A)
    rows = torch.arange(m, device="cuda").repeat_interleave(n // 2)
    X, G = torch.randn(b, n, device="cuda", generator=g), torch.randn(b, m, device="cuda", generator=g).bfloat16()
    ck = H.hss_mx_quantize(X, "int8")
    X64, Gt = H.hss_mx_dequantize(ck, torch.float32).double(), G.double().t().contiguous()
    at = (rows, cols.long())
    err = (H.hss_grad_ckpt(A, ck, G, dU=False, dVt=False)["dS"].double() - (Gt @ X64)[at]).abs()
    assert torch.all(err <= (3 * b + 2) * U24 * (Gt.abs() @ X64.abs())[at])


def test_noalloc_calls_of_both_kinds_in_turn(H):
    """HSS_MX4 calls between the decode kernel's calls, on the library's own
    scratch: each gives the bits of the call with a workspace, call after call."""
    import torch
    A, _, _, _ = _layer(H, 512, 1024, 32, 5, 0.01)
    W = torch.randn(700, 1024, device="cuda").bfloat16()
    sp = H.hss_split(W, "csr")
    B = H.HSSMatrix.from_split(sp, U=torch.randn(700, 40, device="cuda").bfloat16(),
                               Vt=torch.randn(40, 1024, device="cuda").bfloat16())
    for b in (1, 9, 40):
        X = torch.randn(b, 1024, device="cuda").bfloat16()
        want = [H.hss_apply(M, X) for M in (A, B)]
        for _ in range(3):
            for M, w in zip((A, B), want):
                y = torch.empty_like(w)
                assert torch.equal(H.hss_apply_noalloc(M, X, y), w)


def test_two_streams_with_their_own_workspaces(H):
    """Calls that overlap on two streams, each with its own workspace."""
    import torch
    A, _, _, _ = _layer(H, 1024, 2048, 32, 6, 0.01)
    for b in (3, 12, 100, 400):
        X = [torch.randn(b, 2048, device="cuda").bfloat16() for _ in range(2)]
        want = [H.hss_apply(A, x) for x in X]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = [None, None]
        for _ in range(4):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[i] = H.hss_apply(A, X[i])
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_long_rows(H):
    """Rows past the one-pass sizes: 65,600 columns (X of one column beyond the
    vector route's LDS), and S in 16-bit columns up to the largest index."""
    import torch
    for m, n, b, c16 in ((33, 65600, 1, False), (40, 65536, 3, True), (20, 40000, 20, True)):
        A, W, _, _ = _layer(H, m, n, 8, 9, 0.001, col16=c16)
        X = torch.randn(b, n, device="cuda").bfloat16()
        X64 = X.double()
        T = X64 @ A.Vt.double().t().contiguous()
        ref = X64 @ W.t().contiguous() + T @ A.U.double().t().contiguous()
        N = X64.abs() @ W.abs().t().contiguous() + \
            (X64.abs() @ A.Vt.double().abs().t().contiguous()) @ A.U.double().abs().t().contiguous()
        err = (H.hss_apply(A, X).double() - ref).abs()
        assert torch.all(err <= 2.0 ** -8 * ref.abs() + ((2 * n + 18) * U24 + 2.0 ** -16) * N)


def test_quantise_large(H):
    """More groups than one pass of the grid: values against the plain rule in
    float64, and the decoded values' half-step bound."""
    import torch
    W = torch.randn(9000, 4100, device="cuda") * 0.02
    for fmt, bits, q in (("fp4", 2, 2), ("int8", 7, 6)):
        x, res = H.hss_mx_quantize(W, fmt, residual=True)
        D = H.hss_mx_dequantize(x, torch.float32)
        assert torch.equal(W - D, res)
        s = 2.0 ** (x.scales.double() - 127 - (0 if fmt == "fp4" else 6))
        s = s.repeat_interleave(32, 1)[:, :4100]
        half = torch.maximum(2.0 ** torch.floor(torch.log2(W.double().abs().clamp(min=1e-30))), s) / 4 \
            if fmt == "fp4" else s / 2
        assert torch.all((W.double() - D.double()).abs() <= half * (1 + 2.0 ** -40))


def test_kept_weights_are_not_written(H):
    """A call leaves its operands as they were."""
    import torch
    A, _, _, _ = _layer(H, 300, 777, 24, 8, 0.02)
    At = H.hss_transposed_layer(A)
    for b in (1, 8, 60, 300):
        X, G = torch.randn(b, 777, device="cuda").bfloat16(), torch.randn(b, 300, device="cuda").bfloat16()
        ck = H.hss_mx_quantize(X, "int8")
        held = [A.mx.codes, A.mx.scales, A.values, A.U, A.Vt, A.row_ptr, A.col_idx, X, G, ck.codes, ck.scales]
        before = [t.clone() for t in held]
        H.hss_apply(A, X), H.hss_apply(At, G), H.hss_grad_ckpt(A, ck, G)
        assert all(torch.equal(a, b_) for a, b_ in zip(held, before))


@pytest.mark.parametrize("b", [1, 8, 100, 200, 300])
def test_arrays_past_2_gib(H, b):
    """A dense part whose bf16 copy has more than 2^31 bytes, both directions
    (beyond 256 columns such a copy is made): a sample of the outputs, the last
    ones among them, in float64.  S in the last rows."""
    import torch
    m, n, r = 33001, 32800, 8
    g = torch.Generator(device="cuda").manual_seed(b)
    ng = n // 32
    codes = torch.randint(0, 256, (m, 16 * ng), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(118, 122, (m, ng), dtype=torch.uint8, device="cuda", generator=g)
    rp = torch.zeros(m + 1, dtype=torch.int32, device="cuda")
    rp[-2:] = torch.tensor([2, 5], device="cuda")
    cols = torch.tensor([0, n - 1, 5, 6, n - 1], device="cuda")
    srow = torch.tensor([m - 2, m - 2, m - 1, m - 1, m - 1], device="cuda")
    vals = torch.tensor([0.5, -0.25, 0.75, 1.0, -1.5], device="cuda").bfloat16()
    for p in range(5):                                            # D kept zero under S
        at = codes[srow[p], cols[p] // 32 * 16 + cols[p] % 32 // 2]
        at &= 0xF0 if cols[p] % 2 == 0 else 0x0F
    U = (0.05 * torch.randn(m, r, device="cuda", generator=g)).bfloat16()
    Vt = (0.05 * torch.randn(r, n, device="cuda", generator=g)).bfloat16()
    A = H.HSSMatrix("csr", m, n, torch.bfloat16, U=U, Vt=Vt, row_ptr=rp, col_idx=cols.int(), values=vals, nnz=5,
                    mx=H.MXTensor("fp4", m, n, codes, scales))

    def values(rows, gs):                                         # D[rows][columns of the groups gs]
        by = codes.view(m, ng, 16)[rows][:, gs]
        q = torch.stack((by & 15, by >> 4), -1).flatten(2)
        ex, frac = ((q >> 1) & 3).double(), (q & 1).double()
        v = torch.where(ex == 0, 0.5 * frac, (1 + 0.5 * frac) * 2.0 ** (ex - 1)) * (1 - 2 * (q >> 3).double())
        return (v * 2.0 ** (scales[rows][:, gs].double() - 127)[..., None]).flatten(1)

    for trans in (False, True):
        M = H.hss_transposed_layer(A) if trans else A
        X = torch.randn(b, M.n, device="cuda", generator=g).bfloat16()
        Y = H.hss_apply(M, X)
        X64 = X.double()
        if trans:
            gs = torch.tensor([0, 1, 500, ng - 2, ng - 1], device="cuda")
            at = (gs[:, None] * 32 + torch.arange(32, device="cuda")).flatten()
            W = values(torch.arange(m, device="cuda"), gs).t().contiguous()
            for p in range(5):
                W[at == cols[p], srow[p]] += vals[p].double()
            left, right = U.double(), Vt.double()[:, at].contiguous()
        else:
            at = torch.cat((torch.arange(0, m, 701, device="cuda"), torch.arange(m - 9, m, device="cuda")))
            W = values(at, torch.arange(ng, device="cuda"))
            for p in range(5):
                W[at == srow[p], cols[p]] += vals[p].double()
            left, right = Vt.double().t().contiguous(), U.double()[at].t().contiguous()
        Wt = W.t().contiguous()
        ref = X64 @ Wt + (X64 @ left) @ right
        N = X64.abs() @ Wt.abs() + (X64.abs() @ left.abs()) @ right.abs()
        err = (Y[:, at].double() - ref).abs()
        assert torch.all(err <= 2.0 ** -8 * ref.abs() + ((2 * M.n + 2 * r + 2) * U24 + 2.0 ** -16) * N)
