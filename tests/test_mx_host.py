"""Microscaled formats without a GPU: the oracle's encoding pinned by hand
values, by the half-step bound and by brute force, and the library's host-side
refusals (every call below fails its argument checks before any device work)."""
import ctypes

import numpy as np
import pytest

import hss_synth as syn
import oracle as O

FAKE = 1 << 20  # never dereferenced


@pytest.fixture(scope="module")
def hl():
    import sparse_rank_linear_hss_amd as h
    return h


# ---------------------------------------------------------------------------
# The oracle's encoding
# ---------------------------------------------------------------------------

def test_fp4_hand_group():
    """Largest magnitude 6: scale 1, every grid value kept, ties to the even code."""
    w = np.zeros((1, 32))
    w[0, :12] = [0, 0.5, -1, 1.5, 2, -3, 4, 6, 0.25, 0.75, 2.5, 5]
    codes, scales = O.mx_encode(w, "fp4")
    assert scales.tolist() == [[127]]
    nib = [c for byte in codes[0, :6] for c in (byte & 15, byte >> 4)]
    assert nib == [0, 1, 8 | 2, 3, 4, 8 | 5, 6, 7, 0, 2, 4, 6]
    assert O.mx_decode(codes, scales, 12, "fp4").tolist() == [[0, 0.5, -1, 1.5, 2, -3, 4, 6, 0, 1, 2, 4]]


def test_largest_magnitude_carries_into_the_next_exponent():
    """7 is halfway between 6 and 8: it takes 8 = 4 * 2; just below it takes 6.
    127.5 / 64 takes 128 / 64 = 64 / 32; just below 127 / 64."""
    for a, scale, value in ((7.0, 128, 8.0), (np.nextafter(7.0, 0), 127, 6.0)):
        codes, scales = O.mx_encode(np.full((1, 1), a), "fp4")
        assert scales[0, 0] == scale and O.mx_decode(codes, scales, 1, "fp4")[0, 0] == value
    for a, scale, value in ((127.5 / 64, 128, 2.0), (np.nextafter(127.5 / 64, 0), 127, 127 / 64)):
        codes, scales = O.mx_encode(np.full((1, 1), a), "int8")
        assert scales[0, 0] == scale and O.mx_decode(codes, scales, 1, "int8")[0, 0] == value


def test_int8_hand_group():
    w = np.zeros((1, 5))
    w[0] = [1.0, -1.984375, 0.5 / 64, 1.5 / 64, -2.5 / 64]
    codes, scales = O.mx_encode(w, "int8")
    assert scales.tolist() == [[127]] and codes[0, :6].tolist() == [64, -127, 0, 2, -2, 0] and codes.shape == (1, 32)


@pytest.mark.parametrize("fmt", ["fp4", "int8"])
@pytest.mark.parametrize("dtype", [O.F32, O.BF16])
def test_no_value_is_off_by_more_than_half_a_step(fmt, dtype):
    """fp4: half a step is a quarter of the value's power of two (at least a
    quarter of the group's scale); int8: half the group's step."""
    W = O.widen(syn.random_matrix(9, 203, dtype, seed=5, kind="t3"), dtype)
    codes, scales = O.mx_encode(W, fmt)
    D = O.mx_decode(codes, scales, 203, fmt)
    s = np.repeat(2.0 ** (scales.astype(float) - 127), 32, axis=1)[:, :203]
    if fmt == "fp4":
        half = np.maximum(2.0 ** np.floor(np.log2(np.maximum(np.abs(W), 1e-300))), s) / 4
    else:
        half = s / 64 / 2
    assert np.all(np.abs(W - D) <= half)


@pytest.mark.parametrize("dtype", [O.F32, O.BF16])
def test_borders_of_the_exponent_range(dtype):
    big = O.widen(np.array([[0x7F7F0000]], np.uint32).view(np.float32), O.F32)     # bf16's largest
    codes, scales = O.mx_encode(big, "fp4")
    assert scales[0, 0] == 252 and O.mx_decode(codes, scales, 1, "fp4")[0, 0] == 6 * 2.0 ** 125
    codes, scales = O.mx_encode(big, "int8")
    assert scales[0, 0] == 254 and O.mx_decode(codes, scales, 1, "int8")[0, 0] == 127 * 2.0 ** 121
    for fmt, low in (("fp4", 2), ("int8", 7)):
        codes, scales = O.mx_encode(np.array([[2.0 ** -126, 0.0]]), fmt)
        assert scales[0, 0] == low
    codes, scales = O.mx_encode(np.array([[np.nan, 1.0]]), "fp4")
    assert scales[0, 0] == 255 and np.all(np.isnan(O.mx_decode(codes, scales, 2, "fp4")))


# ---------------------------------------------------------------------------
# Refusals of the library
# ---------------------------------------------------------------------------

def test_mx_sizes(hl):
    lib = hl._lib.lib
    c, s = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.hss_mx_sizes(0, 3, 33, ctypes.byref(c), ctypes.byref(s)) == 0 and (c.value, s.value) == (96, 6)
    assert lib.hss_mx_sizes(1, 3, 33, ctypes.byref(c), ctypes.byref(s)) == 0 and (c.value, s.value) == (192, 6)
    INV = hl._lib.HSS_ERR_INVALID_ARG
    for fmt, rows, cols in ((2, 3, 33), (-1, 3, 33), (0, 0, 33), (0, 3, 0), (0, 1 << 26, 1), (1, 65536, 32768)):
        assert lib.hss_mx_sizes(fmt, rows, cols, ctypes.byref(c), ctypes.byref(s)) == INV
    assert lib.hss_mx_sizes(0, 3, 33, None, ctypes.byref(s)) == INV


def test_quantize_rejects_bad_arguments(hl):
    lib, INV = hl._lib.lib, hl._lib.HSS_ERR_INVALID_ARG

    def q(fmt=0, dt=1, rows=4, cols=64, src=FAKE, codes=FAKE * 2, scales=FAKE * 3, res=None):
        return lib.hss_mx_quantize(fmt, dt, rows, cols, src, codes, scales, res, None)

    def d(fmt=0, dt=1, rows=4, cols=64, codes=FAKE * 2, scales=FAKE * 3, dst=FAKE):
        return lib.hss_mx_dequantize(fmt, dt, rows, cols, codes, scales, dst, None)

    for kw in (dict(fmt=2), dict(dt=2), dict(rows=0), dict(cols=-1), dict(rows=1 << 26, cols=1), dict(codes=None),
               dict(scales=None), dict(codes=FAKE * 2 + 8)):
        assert q(**kw) == INV, kw
        assert d(**kw) == INV, kw
    for kw in (dict(src=None), dict(scales=FAKE * 2 + 4), dict(src=FAKE + 1), dict(src=FAKE + 2, dt=0), dict(codes=FAKE + 16),
               dict(scales=FAKE + 100), dict(res=FAKE + 2), dict(res=FAKE * 2 + 2), dict(res=FAKE * 3),
               dict(res=FAKE * 5 + 1)):
        assert q(**kw) == INV, kw
    for kw in (dict(dst=None), dict(dst=FAKE + 1), dict(dst=FAKE * 2), dict(dst=FAKE * 3 - 4)):
        assert d(**kw) == INV, kw


def _mx(hl, **kw):
    s = hl._lib.HssMatrixStruct()
    s.fmt, s.dtype, s.m, s.n, s.r, s.flags, s.nnz = 0, 1, 16, 32, 4, 16, 10
    s.row_ptr = s.col_idx = s.values = FAKE
    s.U, s.Vt = FAKE, FAKE + 4096
    s.dq_codes, s.dq_levels = FAKE * 6, FAKE * 7
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def test_apply_checks_a_microscaled_dense_part(hl):
    lib = hl._lib.lib
    INV, WS, UNS = hl._lib.HSS_ERR_INVALID_ARG, hl._lib.HSS_ERR_WORKSPACE, hl._lib.HSS_ERR_UNSUPPORTED

    def apply(s, b=1, X=FAKE * 8, Y=FAKE * 9, ws=FAKE * 16, wsb=0):
        return lib.hss_apply(ctypes.byref(s), b, X, Y, ws, wsb, None)

    assert apply(_mx(hl)) == WS                                   # valid but for the workspace
    assert apply(_mx(hl, flags=48)) == WS                         # the transposed form
    assert apply(_mx(hl, flags=17)) == WS                         # 16-bit columns
    assert apply(_mx(hl, nnz=0, col_idx=None, values=None, r=0, U=None, Vt=None)) == WS
    assert apply(_mx(hl, flags=32)) == INV                        # transposed without the part
    assert apply(_mx(hl, flags=16 | 2)) == INV                    # two dense parts
    assert apply(_mx(hl, flags=16 | 4)) == INV                    # with the block low-rank form
    assert apply(_mx(hl, fmt=1, nm_values=FAKE, nm_meta=FAKE)) == INV
    assert apply(_mx(hl, dq_codes=None)) == INV
    assert apply(_mx(hl, dq_levels=None)) == INV
    assert apply(_mx(hl, dq_codes=FAKE * 6 + 8)) == INV
    assert apply(_mx(hl, row_ptr=None)) == INV
    assert apply(_mx(hl, dtype=0)) == UNS
    assert apply(_mx(hl, m=1 << 26, n=1)) == INV                  # 32 m bytes of padded rows
    assert apply(_mx(hl, m=1, n=1 << 26)) == INV                  # and of the transposed array
    assert apply(_mx(hl), X=FAKE * 9, Y=FAKE * 9) == INV
    assert apply(_mx(hl), b=2049) == INV
    out = ctypes.c_size_t()
    assert lib.hss_apply_workspace_size(ctypes.byref(_mx(hl)), 4, ctypes.byref(out)) == 0 and out.value > 0
    assert lib.hss_grad_workspace_size(ctypes.byref(_mx(hl)), 4, ctypes.byref(out)) == 0


def test_grad_ckpt_rejects_bad_arguments(hl):
    lib = hl._lib.lib
    INV, WS, UNS = hl._lib.HSS_ERR_INVALID_ARG, hl._lib.HSS_ERR_WORKSPACE, hl._lib.HSS_ERR_UNSUPPORTED

    def grad(s, b=4, codes=FAKE * 8, scales=FAKE * 9, G=FAKE * 10, dS=FAKE * 11, dU=FAKE * 12, dVt=FAKE * 13,
             ws=FAKE * 16, wsb=0):
        return lib.hss_grad_ckpt(ctypes.byref(s), b, codes, scales, G, dS, dU, dVt, ws, wsb, None)

    plain = _mx(hl, flags=0, dq_codes=None, dq_levels=None)
    assert grad(plain) == WS and grad(_mx(hl)) == WS
    assert grad(plain, ws=None, wsb=1 << 30) == WS
    for kw in (dict(codes=None), dict(scales=None), dict(G=None), dict(codes=FAKE * 8 + 8), dict(b=0), dict(b=2049),
               dict(dS=FAKE * 10), dict(dU=FAKE * 8 + 4), dict(dVt=FAKE * 9 + 1), dict(dU=FAKE * 11 + 4)):
        assert grad(plain, **kw) == INV, kw
    assert grad(_mx(hl, flags=0, dtype=0)) == UNS
    assert grad(_mx(hl, flags=2, r=0, U=None, Vt=None)) == UNS     # a per-row table part
    out = ctypes.c_size_t()
    assert lib.hss_grad_ckpt_workspace_size(ctypes.byref(plain), 4, None) == INV
    assert lib.hss_grad_ckpt_workspace_size(ctypes.byref(_mx(hl, flags=0, m=1 << 19, n=8, r=0)), 2048,
                                            ctypes.byref(out)) == UNS


def test_binding_checks(hl):
    import torch
    q = hl.MXTensor.empty("fp4", 3, 33, "cpu")
    assert q.codes.shape == (3, 32) and q.scales.shape == (3, 2)
    assert hl.MXTensor.empty("int8", 3, 33, "cpu").codes.shape == (3, 64)
    with pytest.raises(ValueError):
        hl.MXTensor("fp8", 3, 33, q.codes, q.scales)
    with pytest.raises(ValueError):
        hl.MXTensor("fp4", 3, 65, q.codes, q.scales)
    with pytest.raises(ValueError):
        hl.MXTensor("int8", 3, 33, q.codes, q.scales)
    with pytest.raises(ValueError):
        hl.MXTensor("fp4", 3, 33, q.codes, q.scales.t())
    with pytest.raises(ValueError):
        hl.hss_mx_quantize(torch.zeros(3, 33), "fp4")             # not on a GPU
    with pytest.raises(ValueError):
        hl.HSSMatrix("csr", 33, 3, torch.bfloat16, mx=q)          # shapes swapped
    with pytest.raises(ValueError):
        hl.HSSMatrix("csr", 3, 33, torch.bfloat16, mx_t=True)
    A = hl.HSSMatrix("csr", 3, 33, torch.bfloat16, mx=q)
    assert A.nnz == 0 and A.row_ptr.shape == (4,) and hl.hss_apply_workspace_size(A, 5) > 0
    At = hl.HSSMatrix("csr", 33, 3, torch.bfloat16, mx=q, mx_t=True)
    assert At.flags == hl.HSS_MX4 | hl.HSS_MX4_T


def test_binding_refuses_other_devices(hl):
    """A CPU workspace, and a dense part on another device than the rest."""
    import torch
    with pytest.raises(ValueError):
        hl.hss_apply_workspace_init(torch.zeros(4096, dtype=torch.uint8))
    q = hl.MXTensor.empty("fp4", 3, 33, "cpu")
    with pytest.raises(ValueError):
        hl.HSSMatrix("csr", 3, 33, torch.bfloat16, mx=q, U=torch.empty(3, 2, dtype=torch.bfloat16, device="meta"),
                     Vt=torch.empty(2, 33, dtype=torch.bfloat16, device="meta"))


def test_group_takes_one_kind_of_matrix(hl):
    """HSS_MX4 matrices are grouped among themselves (they leave dense data where
    others keep state)."""
    lib, INV = hl._lib.lib, hl._lib.HSS_ERR_INVALID_ARG
    P = ctypes.POINTER(hl._lib.HssMatrixStruct)
    out = ctypes.c_size_t()
    mx, plain = _mx(hl), _mx(hl, flags=0, dq_codes=None, dq_levels=None)
    for mats, want in (((mx, mx), 0), ((mx, plain), INV), ((plain, mx), INV), ((mx, _mx(hl, flags=48)), INV)):
        arr = (P * 2)(*[ctypes.pointer(s) for s in mats])
        assert lib.hss_apply_group_workspace_size(arr, 2, 1, ctypes.byref(out)) == want


@pytest.fixture
def bound(hl, monkeypatch):
    """The binding with its library calls recorded, CPU tensors standing for the
    current device's (their index is -1) and `elsewhere` for another device's."""
    import torch

    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 1

    calls = []

    class Lib:
        def __getattr__(self, name):
            real = getattr(hl._lib.lib, name)
            if name.endswith("_size") or name == "hss_noalloc_scratch_bytes":
                return real
            return lambda *a: calls.append(name) or 0

    monkeypatch.setattr(hl, "lib", Lib())
    monkeypatch.setattr(hl, "_current_device", lambda: -1)
    monkeypatch.setattr(hl, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(hl, "_index", lambda t: t.get_device())
    return calls, lambda t: t.as_subclass(Elsewhere)


def _cpu_layer(hl, kind):
    import torch
    bf = torch.bfloat16
    U, Vt = torch.zeros(3, 2, dtype=bf), torch.zeros(2, 33, dtype=bf)
    if kind == "mx":
        return hl.HSSMatrix("csr", 3, 33, bf, U=U, Vt=Vt, mx=hl.MXTensor.empty("fp4", 3, 33, "cpu"))
    return hl.HSSMatrix("csr", 3, 33, bf, U=U, Vt=Vt, row_ptr=torch.zeros(4, dtype=torch.int32))


@pytest.mark.parametrize("kind", ["mx", "csr"])
def test_applies_refuse_outputs_and_workspaces_that_do_not_fit(hl, bound, kind):
    """What the kernels would write or read out of range: Y of another shape,
    type, layout or device, a workspace on another device or with strides, and
    a matrix that lies elsewhere than X."""
    import torch
    calls, elsewhere = bound
    bf = torch.bfloat16
    A = _cpu_layer(hl, kind)
    X, Y = torch.zeros(5, 33, dtype=bf), torch.zeros(5, 3, dtype=bf)
    size = max(hl.hss_apply_workspace_size(A, 5), hl.hss_apply_group_workspace_size([A, A], 5))
    ws = torch.zeros(size, dtype=torch.uint8)
    hl.hss_apply(A, X, Y, ws), hl.hss_apply_noalloc(A, X, Y), hl.hss_apply_group([A, A], X, [Y, Y.clone()], ws)
    assert calls == ["hss_apply", "hss_apply_noalloc", "hss_apply_group"]
    bad_y = [torch.zeros(5, 2, dtype=bf), torch.zeros(3, 5, dtype=bf), torch.zeros(4, 3, dtype=bf), torch.zeros(15, dtype=bf),
             torch.zeros(5, 3), torch.zeros(3, 5, dtype=bf).t(), torch.zeros(5, 6, dtype=bf)[:, ::2], elsewhere(Y)]
    for y in bad_y:
        for call in (lambda: hl.hss_apply(A, X, y, ws), lambda: hl.hss_apply_noalloc(A, X, y),
                     lambda: hl.hss_apply_group([A, A], X, [Y, y], ws)):
            with pytest.raises(ValueError):
                call()
    for w in (elsewhere(ws), torch.zeros(1, dtype=torch.uint8).expand(size), torch.zeros(2 * size, dtype=torch.uint8)[::2]):
        for call in (lambda: hl.hss_apply(A, X, Y, w), lambda: hl.hss_apply_group([A, A], X, [Y, Y.clone()], w)):
            with pytest.raises(ValueError):
                call()
    for x in (torch.zeros(5, 32, dtype=bf), torch.zeros(5, 33), torch.zeros(33, dtype=bf), torch.zeros(33, 5, dtype=bf).t()):
        with pytest.raises(ValueError):
            hl.hss_apply(A, x, Y, ws)
    with pytest.raises(ValueError):
        hl.hss_apply_group([A, A], X, [Y], ws)
    A.index = 1                                                    # the matrix elsewhere
    for call in (lambda: hl.hss_apply(A, X, Y, ws), lambda: hl.hss_apply_noalloc(A, X, Y),
                 lambda: hl.hss_apply_group([A], X, [Y], ws)):
        with pytest.raises(ValueError):
            call()
    assert len(calls) == 3


def test_a_matrix_over_two_devices_has_no_device(hl, bound):
    import torch
    calls, elsewhere = bound
    bf = torch.bfloat16
    A = hl.HSSMatrix("csr", 3, 33, bf, U=elsewhere(torch.zeros(3, 2, dtype=bf)), Vt=torch.zeros(2, 33, dtype=bf),
                     row_ptr=torch.zeros(4, dtype=torch.int32))
    assert A.index is None
    with pytest.raises(ValueError):
        hl.hss_apply_noalloc(A, torch.zeros(1, 33, dtype=bf), torch.zeros(1, 3, dtype=bf))
    assert not calls


def test_gradients_refuse_inputs_and_workspaces_elsewhere(hl, bound, monkeypatch):
    import torch
    calls, elsewhere = bound
    monkeypatch.setattr(hl, "_dev", lambda t: t.device)
    monkeypatch.setattr(hl, "_stream", lambda device: 0)
    bf = torch.bfloat16
    A = _cpu_layer(hl, "csr")
    X, G, ck = torch.zeros(5, 33, dtype=bf), torch.zeros(5, 3, dtype=bf), hl.MXTensor.empty("int8", 5, 33, "cpu")
    hl.hss_grad(A, X, G), hl.hss_grad_ckpt(A, ck, G)
    assert calls == ["hss_grad", "hss_grad_ckpt"]
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    calls_in = [lambda A=A: hl.hss_grad(A, X, elsewhere(G)), lambda A=A: hl.hss_grad(A, X, G, ws=elsewhere(ws)),
                lambda A=A: hl.hss_grad(A, X, G, ws=ws[:1].expand(1 << 20)),
                lambda A=A: hl.hss_grad_ckpt(A, ck, G, ws=elsewhere(ws)),
                lambda A=A: hl.hss_grad_ckpt(A, ck, G, ws=ws[:1].expand(1 << 20))]
    A.index = 1
    calls_in += [lambda: hl.hss_grad(A, X, G), lambda: hl.hss_grad_ckpt(A, ck, G)]
    for k, call in enumerate(calls_in):
        A.index = 1 if k >= 5 else -1
        with pytest.raises(ValueError):
            call()
    assert len(calls) == 2


def test_backward_launches_on_the_device_of_its_tensors(hl, bound, monkeypatch):
    """hss_backward with every tensor on another GPU than the current one: each
    launch of its parts (transposes, workspace, gradients, apply) is made with
    that GPU current."""
    import contextlib

    import torch
    calls, elsewhere = bound
    current, seen = [0], []

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before

    class Lib:
        def __getattr__(self, name):
            real = getattr(hl._lib.lib, name)
            if name.endswith("_size") or name in ("hss_csr_transpose", "hss_apply_group_workspace_size"):
                return real
            return lambda *a: seen.append((name, current[0])) or 0

    new = lambda *a, dtype=None, device=None: elsewhere(torch.zeros(*a, dtype=dtype))
    monkeypatch.setattr(hl, "lib", Lib())
    monkeypatch.setattr(hl, "_current_device", lambda: current[0])
    monkeypatch.setattr(hl, "_stream", lambda dev: 0)
    monkeypatch.setattr(hl, "_dev", lambda t: t.device)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch, "empty", new)
    monkeypatch.setattr(torch, "from_numpy", lambda a, f=torch.from_numpy: elsewhere(f(a)))
    bf = torch.bfloat16
    A = hl.HSSMatrix("csr", 3, 33, bf, U=elsewhere(torch.zeros(3, 2, dtype=bf)), Vt=elsewhere(torch.zeros(2, 33, dtype=bf)),
                     row_ptr=elsewhere(torch.tensor([0, 1, 1, 2], dtype=torch.int32)),
                     col_idx=elsewhere(torch.tensor([4, 7], dtype=torch.int32)), values=elsewhere(torch.zeros(2, dtype=bf)))
    hl.hss_backward(A, elsewhere(torch.zeros(5, 33, dtype=bf)), elsewhere(torch.zeros(5, 3, dtype=bf)))
    names = [n for n, _ in seen]
    for name in ("hss_gather_values", "hss_transpose", "hss_grad", "hss_apply_workspace_init", "hss_apply"):
        assert name in names
    assert all(index == 1 for _, index in seen), seen
    assert current == [0]


SIZES = [(4096, 4096, 64, 1000, 16), (4096, 4096, 0, 0, 16), (4096, 4096, 64, 1000, 48), (8192, 8192, 512, 1000, 16),
         (512, 4096, 0, 0, 16), (11000, 640, 24, 3, 16), (4096, 11008, 64, 5, 48), (33, 700, 900, 7, 16), (1, 1, 0, 0, 16)]


@pytest.mark.parametrize("case", SIZES, ids=["x".join(map(str, c)) for c in SIZES])
def test_a_workspace_serves_every_smaller_batch(hl, case):
    """hss_apply_workspace_size never goes down as b goes up, for one matrix and
    for a group, and is never less than a call asks for."""
    lib, WS = hl._lib.lib, hl._lib.HSS_ERR_WORKSPACE
    m, n, r, nnz, flags = case
    s = _mx(hl, m=m, n=n, r=r, nnz=nnz, flags=flags)
    P = ctypes.POINTER(hl._lib.HssMatrixStruct)
    pair = (P * 2)(ctypes.pointer(s), ctypes.pointer(_mx(hl, m=2 * m, n=n, r=0, nnz=0, flags=flags)))
    out, last, last_pair = ctypes.c_size_t(), 0, 0
    for b in range(1, 2049):
        assert lib.hss_apply_workspace_size(ctypes.byref(s), b, ctypes.byref(out)) == 0
        assert out.value >= last, b
        last = out.value
        if b % 16 in (0, 1):
            assert lib.hss_apply_group_workspace_size(pair, 2, b, ctypes.byref(out)) == 0
            assert out.value >= max(last, last_pair), b
            last_pair = out.value
    assert lib.hss_apply(ctypes.byref(s), 2048, FAKE * (1 << 14), FAKE * (1 << 16), FAKE, 32768 - 1, None) == WS


@pytest.mark.parametrize("case", [(4096, 4096, 64, 800000), (8192, 8192, 128, 2000000), (1501, 2777, 41, 80000), (64, 11008, 40, 7000)],
                         ids=lambda c: f"{c[0]}x{c[1]}")
def test_a_gradient_workspace_serves_every_smaller_batch(hl, case):
    """hss_grad_ckpt_workspace_size never goes down as b goes up, and does not
    depend on the route of dS."""
    lib, out = hl._lib.lib, ctypes.c_size_t()
    m, n, r, nnz = case
    s = _mx(hl, m=m, n=n, r=r, nnz=nnz, flags=0, dq_codes=None, dq_levels=None)
    sizes = []
    for b in range(1, 2049):
        assert lib.hss_grad_ckpt_workspace_size(ctypes.byref(s), b, ctypes.byref(out)) == 0
        sizes.append(out.value)
    assert sizes == sorted(sizes)
    for route in ("sparse", "dense"):
        with hl.option("grad_ds_route", route):
            for b in (1, 33, 600, 2048):
                assert hl._lib.lib.hss_grad_ckpt_workspace_size(ctypes.byref(s), b, ctypes.byref(out)) == 0
                assert out.value == sizes[b - 1]


def test_transposed_layer_refuses_another_layers(hl):
    import torch
    bf = torch.bfloat16

    def layer(m=3, n=33, r=2, nnz=2, mx=None, mx_t=False):
        rp = torch.zeros(m + 1, dtype=torch.int32)
        rp[-1:] = nnz
        return hl.HSSMatrix("csr", m, n, bf, U=torch.zeros(m, r, dtype=bf), Vt=torch.zeros(r, n, dtype=bf), row_ptr=rp,
                            col_idx=torch.arange(nnz, dtype=torch.int32), values=torch.zeros(nnz, dtype=bf), mx=mx, mx_t=mx_t)

    A = layer()
    q = hl.MXTensor.empty("fp4", 3, 33, "cpu")
    for out in (layer(33, 3), layer(33, 4), layer(33, 3, r=3), layer(33, 3, nnz=3), layer(33, 3, mx=q, mx_t=True), A):
        if out is not A:
            out.perm_from_s = torch.zeros(2, dtype=torch.int32)
        if (out.m, out.n, out.r, out.nnz) == (33, 3, 2, 2) and out.mx is None:
            out.index = 1                                         # on another device
        with pytest.raises(ValueError):
            hl.hss_transposed_layer(A, out=out)


def test_matrices_refuse_arrays_that_do_not_fit(hl):
    """Index arrays of 64 bits, short or strided arrays and values of another
    type would be read out of range or as other numbers."""
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    good = dict(row_ptr=torch.zeros(4, dtype=i32), col_idx=torch.zeros(5, dtype=i32), values=torch.zeros(5, dtype=bf))
    hl.HSSMatrix("csr", 3, 33, bf, **good)
    hl.HSSMatrix("csr", 3, 33, bf, row_ptr=good["row_ptr"])
    hl.HSSMatrix("csr", 3, 33, bf, **{**good, "col_idx": torch.zeros(5, dtype=torch.int16)})
    for bad in (dict(row_ptr=torch.zeros(4, dtype=torch.int64)), dict(row_ptr=torch.zeros(3, dtype=i32)), dict(row_ptr=None),
                dict(col_idx=torch.zeros(5, dtype=torch.int64)), dict(col_idx=torch.zeros(4, dtype=i32)), dict(col_idx=None),
                dict(col_idx=torch.zeros(10, dtype=i32)[::2]), dict(values=torch.zeros(5)), dict(nnz=6),
                dict(values=torch.zeros(10, dtype=bf)[::2])):
        with pytest.raises(ValueError):
            hl.HSSMatrix("csr", 3, 33, bf, **{**good, **bad})
    nm = dict(nm_values=torch.zeros(3, 18, dtype=bf), nm_meta=torch.zeros(3, 2, dtype=i32))
    hl.HSSMatrix("2:4", 3, 36, bf, **nm)
    for bad in (dict(nm_values=None), dict(nm_values=torch.zeros(3, 18)), dict(nm_values=torch.zeros(3, 17, dtype=bf)),
                dict(nm_meta=torch.zeros(3, 1, dtype=i32)), dict(nm_meta=torch.zeros(3, 2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            hl.HSSMatrix("2:4", 3, 36, bf, **{**nm, **bad})


def test_transposes_and_gathers_refuse_what_does_not_fit(hl, bound, monkeypatch):
    import torch
    calls, elsewhere = bound
    monkeypatch.setattr(hl, "_stream", lambda device: 0)
    t, perm = torch.zeros(4, 6), torch.zeros(3, dtype=torch.int32)
    hl.hss_transpose(t), hl.hss_gather_values(t, perm)
    assert calls == ["hss_transpose", "hss_gather_values"]
    for bad in (t.t(), t[:, ::2], t[0], t.half(), torch.zeros(1, 6).expand(4, 6)):
        with pytest.raises(ValueError):
            hl.hss_transpose(bad)
    for v, p in ((t, perm.long()), (t, elsewhere(perm)), (t, perm[:1].expand(3)), (t.t(), perm), (t.int(), perm)):
        with pytest.raises(ValueError):
            hl.hss_gather_values(v, p)
    assert len(calls) == 2


def test_calls_refuse_cpu_tensors(hl):
    """With a ValueError, whether or not the machine has a GPU."""
    import torch
    bf = torch.bfloat16
    A = _cpu_layer(hl, "mx")
    X, G, Y = torch.zeros(1, 33, dtype=bf), torch.zeros(1, 3, dtype=bf), torch.zeros(1, 3, dtype=bf)
    ck = hl.MXTensor.empty("int8", 1, 33, "cpu")
    for call in (lambda: hl.hss_apply(A, X), lambda: hl.hss_apply(A, X, Y), lambda: hl.hss_apply_noalloc(A, X, Y),
                 lambda: hl.hss_apply_group([A], X), lambda: hl.hss_grad(A, X, G), lambda: hl.hss_grad_ckpt(A, ck, G),
                 lambda: hl.hss_transpose(X), lambda: hl.hss_gather_values(X, torch.zeros(1, dtype=torch.int32)),
                 lambda: hl.hss_mx_quantize(X), lambda: hl.hss_mx_dequantize(ck), lambda: hl.hss_split(X)):
        with pytest.raises(ValueError):
            call()
