"""HSS_MX4 applies on every kernel variant that a small or middle batch takes,
and where S falls on non-zeros of D: values against float64 on the GPU.

Bounds as in test_gpu_mx.py, u = 2^-24, N the sum of magnitudes:
    |err| <= 2^-8 |Y| + (1 + 2^-8) (((2 n + 2 r + 2) u + 2^-16) N + R)
R = 2^-8 |X| |S + D|^T over the places where both are non-zero, for more than 256
columns (the sum is rounded to bf16 there), else 0.  Up to four columns T stays
in fp32, which the 2^-16 covers."""
import pytest

from test_gpu_mx_large import U24, _layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def H():
    import sparse_rank_linear_hss_amd as h
    return h


def _x(b, n, seed, shift=0):
    """Normal values; shift: that many elements past a 16-byte boundary."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.randn(b * n + 8, device="cuda", generator=g).bfloat16()
    return buf[shift:shift + b * n].view(b, n)


def _check(H, A, W, X, met=None):
    """One apply into guarded memory against X (W + U V^T)^T; the same bits again."""
    import torch
    b, n, m, r = X.shape[0], A.n, A.m, A.r
    out = torch.full((b * m + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = out[8:8 + b * m].view(b, m)
    H.hss_apply(A, X, Y)
    assert torch.all(out[:8] == 7) and torch.all(out[8 + b * m:] == 7)
    X64, Wt = X.double(), W.t().contiguous()
    ref, N = X64 @ Wt, X64.abs() @ Wt.abs()
    if r:
        V, Ut = A.Vt.double().t().contiguous(), A.U.double().t().contiguous()
        ref += (X64 @ V) @ Ut
        N += (X64.abs() @ V.abs()) @ Ut.abs()
    rest = ((2 * n + 2 * r + 2) * U24 + 2.0 ** -16) * N
    if met is not None and b > 256:
        rest += 2.0 ** -8 * (X64.abs() @ met.t().contiguous())
    bound = 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * rest
    err = (Y.double() - ref).abs()
    assert torch.all(err <= bound), float((err / bound.clamp(min=1e-300)).max())
    assert torch.equal(H.hss_apply(A, X), Y)


# One to four columns on the vector units: two and four rows a wave, whole and
# ragged rows of X and U, rows of S of more than 64 entries, b = 3 in a kernel of four
GEMV = [(1030, 1024, 64, 0.1), (1031, 1027, 37, 0.02), (8195, 4100, 0, 0.003), (9001, 1027, 37, 0.01), (8200, 1024, 64, 0.0),
        (8193, 2056, 0, 0.09), (5, 1500, 3, 0.2), (12290, 1024, 64, 0.08), (12801, 1027, 37, 0.01)]


@pytest.mark.parametrize("b", [1, 2, 3, 4])
@pytest.mark.parametrize("case", GEMV, ids=[f"{c[0]}x{c[1]}-r{c[2]}" for c in GEMV])
def test_vector_route(H, case, b):
    m, n, r, density = case
    A, W, _, _ = _layer(H, m, n, r, m + n + b, density, col16=b % 2 == 0)
    _check(H, A, W, _x(b, n, b))
    _check(H, A, W, _x(b, n, b, shift=3))


# Two to sixteen columns on the matrix cores.  D alone reads X's own rows where they
# are aligned and short, else (or with S or U) a copy in operand order; 4 and 8
# waves a block; 1 to 6 chunks of 128 columns a wave in flight, and several batches.
SKINNY_N = [8, 120, 128, 136, 512, 640, 1000, 1536, 2176, 2560, 3336, 4096, 5000, 5120, 5128, 6152, 7000]


@pytest.mark.parametrize("kind", ["D", "all"])
@pytest.mark.parametrize("n", SKINNY_N)
def test_skinny_route(H, n, kind):
    for m, b in ((40, 5), (100, 16), (8300, 13) if n <= 1536 else (531, 11)):
        r, density = (0, 0.0) if kind == "D" else (n % 90 + 1, 0.02)
        A, W, _, _ = _layer(H, m, n, r, m + n + b, density, col16=b == 5)
        _check(H, A, W, _x(b, n, b))
    _check(H, A, W, _x(7, n, 7, shift=1))


# Outputs written straight from the tiles (one K split, no S): rows of whole
# 16-byte pieces, and ragged ones
@pytest.mark.parametrize("r", [0, 24, 33])
@pytest.mark.parametrize("b", [17, 33, 70, 130, 200, 256])
@pytest.mark.parametrize("shape", [(200, 264), (264, 200), (136, 72), (129, 203)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_middle_route_writes_from_its_tiles(H, shape, b, r):
    m, n = shape
    A, W, _, _ = _layer(H, m, n, r, m + b + r, 0.0)
    _check(H, A, W, _x(b, n, b))
    At = H.hss_transposed_layer(A)
    _check(H, At, W.t(), _x(b, m, b))


def _meeting(H, m, n, r, seed, density, col16):
    """S on non-zeros of D: the layer, S + D, and |S + D| where both are non-zero."""
    import torch
    A0, W0, _, _ = _layer(H, m, n, r, seed, 0.0)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    mask = torch.rand(m, n, device="cuda", generator=g) < density
    rows, cols = mask.nonzero(as_tuple=True)
    values = (0.1 * torch.randn(len(rows), device="cuda", generator=g)).bfloat16()
    rp = torch.zeros(m + 1, dtype=torch.int32, device="cuda")
    rp[1:] = mask.sum(1).cumsum(0).int()
    W = W0.clone()
    W[rows, cols] += values.double()
    met = torch.where(mask & (W0 != 0), W.abs(), 0.0)
    A = H.HSSMatrix("csr", m, n, torch.bfloat16, U=A0.U, Vt=A0.Vt, row_ptr=rp, col_idx=cols.int(), values=values,
                    nnz=len(cols), mx=A0.mx)
    return (A.with_col16() if col16 else A), W, met


@pytest.mark.parametrize("col16", [False, True], ids=["int32", "uint16"])
@pytest.mark.parametrize("b", [1, 3, 9, 40, 256, 257, 300, 1024])
def test_sparse_entries_on_the_dense_part(H, b, col16):
    """Their sum counts, in both directions; exact up to 256 columns, rounded to
    bf16 beyond, where they meet and nowhere else."""
    m, n, r = 520, 1100, 20
    A, W, met = _meeting(H, m, n, r, b, 0.05, col16)
    assert int((met > 0).sum()) > 20000
    _check(H, A, W, _x(b, n, b), met)
    _check(H, H.hss_transposed_layer(A), W.t(), _x(b, m, b), met.t())
