"""Adapters without a GPU: the oracle pinned by hand values and by differences,
workspace sizes, and the library's refusals (every call below fails its argument
checks before any device work)."""
import ctypes

import numpy as np
import pytest

import oracle as O

FAKE = 1 << 28  # never dereferenced


@pytest.fixture(scope="module")
def hl():
    import sparse_rank_linear_hss_amd as h
    return h


# ---------------------------------------------------------------------------
# The oracle
# ---------------------------------------------------------------------------

def test_by_hand():
    U = np.array([[[1.0], [2.0]], [[0.0], [-1.0]]])                 # 2 adapters, m = 2, r = 1
    Vt = np.array([[[1.0, 0.0, 1.0]], [[0.0, 3.0, 0.0]]])           # n = 3
    X = np.array([[1.0, 2.0, 3.0], [1.0, 2.0, 3.0], [1.0, 2.0, 3.0], [5.0, 5.0, 5.0]])
    ids, scale, base = [1, 0, -1, 7], [0.5, 2.0], np.full((4, 2), 10.0)
    Y = O.adapters_apply(U, Vt, scale, X, ids, base)
    assert Y.tolist() == [[10.0, -2.0], [12.0, 14.0], [10.0, 10.0], [10.0, 10.0]]
    G = np.array([[0.0, 1.0], [1.0, 1.0], [9.0, 9.0], [9.0, 9.0]])
    dX, dU, dVt = O.adapters_grad(U, Vt, scale, X, G, ids)
    assert dX.tolist() == [[0.0, -6.0, 0.0], [1.5, 0.0, 1.5], [0.0] * 3, [0.0] * 3]
    assert dU.tolist() == [[[2.0], [2.0]], [[0.0], [12.0]]]
    assert dVt.tolist() == [[[1.5, 3.0, 4.5]], [[-2.0, -4.0, -6.0]]]


def test_gradients_are_the_differences():
    """Y is linear in each argument: central differences of sum(G Y) are exact."""
    rng = np.random.default_rng(1)
    L, m, n, r, b = 3, 5, 7, 2, 9
    U, Vt, X = rng.standard_normal((L, m, r)), rng.standard_normal((L, r, n)), rng.standard_normal((b, n))
    G, scale, ids = rng.standard_normal((b, m)), rng.standard_normal(L), rng.integers(-1, L - 1, b)
    got = O.adapters_grad(U, Vt, scale, X, G, ids)

    def loss(x, u, v):
        return float(np.sum(G * O.adapters_apply(u, v, scale, x, ids)))

    for k, grad in enumerate(got):
        args = [X, U, Vt]
        for at in np.ndindex(*args[k].shape):
            ends = []
            for s in (0.5, -0.5):
                moved = [a.copy() for a in args]
                moved[k][at] += s
                ends.append(loss(*moved))
            assert abs(ends[0] - ends[1] - grad[at]) < 1e-9
    assert not got[1][L - 1].any() and not got[2][L - 1].any()      # no row has the last adapter


# ---------------------------------------------------------------------------
# Refusals
# ---------------------------------------------------------------------------

def _bank(hl, **kw):
    s = hl._lib.HssAdaptersStruct(dtype=1, m=96, n=64, r=8, count=3, U=FAKE, Vt=2 * FAKE, scale=3 * FAKE)
    for k, x in kw.items():
        setattr(s, k, x)
    return s


APPLY = dict(b=5, X=4 * FAKE, ids=5 * FAKE, base=6 * FAKE, Y=7 * FAKE, ws=8 * FAKE, size=1 << 24)
GRAD = dict(b=5, X=4 * FAKE, G=9 * FAKE, ids=5 * FAKE, base=6 * FAKE, dX=7 * FAKE, dU=10 * FAKE, dVt=11 * FAKE,
            ws=8 * FAKE, size=1 << 24)


def _apply(hl, bank=None, **kw):
    return hl._lib.lib.hss_adapters_apply(ctypes.byref(bank or _bank(hl)), *{**APPLY, **kw}.values(), None)


def _grad(hl, bank=None, **kw):
    return hl._lib.lib.hss_adapters_grad(ctypes.byref(bank or _bank(hl)), *{**GRAD, **kw}.values(), None)


def test_library_refuses(hl):
    INV, WS, UNS = hl._lib.HSS_ERR_INVALID_ARG, hl._lib.HSS_ERR_WORKSPACE, hl._lib.HSS_ERR_UNSUPPORTED
    none = ctypes.POINTER(hl._lib.HssAdaptersStruct)()
    size = ctypes.c_size_t(0)
    lib = hl._lib.lib
    queries = [lambda s, b=5: lib.hss_adapters_workspace_size(s, b, ctypes.byref(size)),
               lambda s, b=5: lib.hss_adapters_grad_workspace_size(s, b, ctypes.byref(size))]
    assert lib.hss_adapters_apply(none, *APPLY.values(), None) == INV
    assert lib.hss_adapters_grad(none, *GRAD.values(), None) == INV
    assert all(q(none) == INV for q in queries)
    assert lib.hss_adapters_workspace_size(ctypes.byref(_bank(hl)), 5, None) == INV
    assert lib.hss_adapters_grad_workspace_size(ctypes.byref(_bank(hl)), 5, None) == INV
    for bad in (dict(dtype=2), dict(m=0), dict(n=-1), dict(r=0), dict(count=0), dict(count=4097), dict(U=None), dict(Vt=None),
                dict(U=FAKE + 1), dict(Vt=FAKE + 1), dict(scale=FAKE + 2), dict(m=1 << 27), dict(n=1 << 30),
                dict(r=1 << 30), dict(m=2 ** 31 - 1, n=2 ** 31 - 1, r=2 ** 31 - 1, count=4096)):
        assert _apply(hl, _bank(hl, **bad)) == INV, bad
        assert _grad(hl, _bank(hl, **bad)) == INV, bad
        assert all(q(ctypes.byref(_bank(hl, **bad))) == INV for q in queries), bad
    for b in (0, -1, 2049):
        assert _apply(hl, b=b) == INV and _grad(hl, b=b) == INV
        assert all(q(ctypes.byref(_bank(hl)), b) == INV for q in queries)
    wide = _bank(hl, m=1 << 20, r=1, count=1)
    assert _apply(hl, wide, b=2048) == INV and _grad(hl, wide, b=2048) == INV     # b m = 2^31
    assert _apply(hl, _bank(hl, dtype=0)) == UNS and _grad(hl, _bank(hl, dtype=0)) == UNS
    y, x, f = 5 * 96 * 2, 5 * 64 * 2, 3 * 8
    for bad in (dict(X=None), dict(ids=None), dict(Y=None), dict(X=FAKE + 1), dict(ids=FAKE + 2), dict(Y=FAKE + 1),
                dict(base=FAKE + 1), dict(Y=4 * FAKE), dict(Y=4 * FAKE + x - 2), dict(Y=FAKE + f * 96 * 2 - 2),
                dict(Y=2 * FAKE + f * 64 * 2 - 2), dict(Y=3 * FAKE + 8), dict(Y=5 * FAKE + 16), dict(base=7 * FAKE + 2),
                dict(base=7 * FAKE + y - 2)):
        assert _apply(hl, **bad) == INV, bad
    for bad in (dict(X=None), dict(G=None), dict(ids=None), dict(dX=FAKE + 1), dict(dU=FAKE * 10 + 2), dict(dVt=FAKE * 11 + 1),
                dict(base=FAKE + 1), dict(G=FAKE + 1), dict(dX=9 * FAKE), dict(dX=4 * FAKE + x - 2), dict(dU=9 * FAKE + y - 4),
                dict(dU=FAKE), dict(dVt=2 * FAKE), dict(dVt=10 * FAKE), dict(dU=11 * FAKE + 4), dict(dX=10 * FAKE + f * 96 * 4 - 2),
                dict(dU=6 * FAKE), dict(dVt=6 * FAKE), dict(base=7 * FAKE + x - 2), dict(dU=5 * FAKE), dict(dVt=3 * FAKE)):
        assert _grad(hl, **bad) == INV, bad
    for kw in (dict(ws=None), dict(ws=FAKE * 8 + 8), dict(size=16)):
        assert _apply(hl, **kw) == WS and _grad(hl, **kw) == WS
    assert _grad(hl, dX=None, dU=None, dVt=None) == hl._lib.HSS_OK              # nothing asked for


def test_ranks_and_columns_have_limits(hl):
    INV = hl._lib.HSS_ERR_INVALID_ARG
    size = ctypes.c_size_t(0)
    for kw, b in ((dict(m=(1 << 28) + 1, n=1, r=1, count=1), 1), (dict(m=1, n=(1 << 28) + 1, r=1, count=1), 1),
                  (dict(m=1, n=1, r=65537, count=1), 1)):
        assert _apply(hl, _bank(hl, **kw), b=b) == INV and _grad(hl, _bank(hl, **kw), b=b) == INV
        for call in ("hss_adapters_workspace_size", "hss_adapters_grad_workspace_size"):
            query = getattr(hl._lib.lib, call)
            assert query(ctypes.byref(_bank(hl, **kw)), b, ctypes.byref(size)) == INV
            kw = {k: x - (x in (65537, (1 << 28) + 1)) for k, x in kw.items()}
            assert query(ctypes.byref(_bank(hl, **kw)), b, ctypes.byref(size)) == 0 and size.value > 0
            kw = {k: x + (x in (65536, 1 << 28)) for k, x in kw.items()}


def test_workspaces_grow_with_the_batch(hl):
    size = ctypes.c_size_t(0)
    for call in ("hss_adapters_workspace_size", "hss_adapters_grad_workspace_size"):
        for m, n, r, count in ((96, 64, 8, 3), (4096, 4096, 16, 1), (11008, 4096, 64, 64), (1, 1, 1, 4096), (300, 5000, 200, 2)):
            got = []
            for b in (1, 2, 15, 16, 17, 63, 64, 65, 66, 128, 500, 2047, 2048):
                s = _bank(hl, m=m, n=n, r=r, count=count)
                assert getattr(hl._lib.lib, call)(ctypes.byref(s), b, ctypes.byref(size)) == 0
                got.append(size.value)
            assert got == sorted(got) and got[0] > 0 and got[-1] < 1 << 28


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
            return real if name.endswith("_size") else lambda *a: calls.append(name) or 0

    monkeypatch.setattr(hl, "lib", Lib())
    monkeypatch.setattr(hl, "_current_device", lambda: -1)
    monkeypatch.setattr(hl, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(hl, "_index", lambda t: t.get_device())
    return calls, lambda t: t.as_subclass(Elsewhere)


def test_banks_refuse_what_does_not_fit(hl, bound):
    import torch
    _, elsewhere = bound
    bf = torch.bfloat16
    z = lambda *k, dt=bf: torch.zeros(*k, dtype=dt)  # noqa: E731
    L = hl.HSSAdapters(z(3, 6, 2), z(3, 2, 5), z(3, dt=torch.float32))
    assert (L.count, L.m, L.n, L.r) == (3, 6, 5, 2)
    for U, Vt, scale in ((z(6, 2), z(3, 2, 5), None), (z(3, 6, 2), z(2, 2, 5), None), (z(3, 6, 2), z(3, 3, 5), None),
                         (z(3, 6, 2), z(3, 2, 5, dt=torch.float32), None), (z(3, 2, 6).transpose(1, 2), z(3, 2, 5), None),
                         (z(3, 6, 2), z(3, 2, 10)[..., ::2], None), (z(3, 6, 2), elsewhere(z(3, 2, 5)), None),
                         (z(3, 6, 2), z(3, 2, 5), z(3)), (z(3, 6, 2), z(3, 2, 5), z(2, dt=torch.float32)),
                         (z(3, 6, 2), z(3, 2, 5), elsewhere(z(3, dt=torch.float32))),
                         (z(3, 6, 2), z(3, 2, 5), z(6, dt=torch.float32)[::2])):
        with pytest.raises(ValueError):
            hl.HSSAdapters(U, Vt, scale)
    with pytest.raises(TypeError):
        hl.HSSAdapters(z(3, 6, 2, dt=torch.float16), z(3, 2, 5, dt=torch.float16))


def test_calls_refuse_what_does_not_fit(hl, bound):
    import torch
    calls, elsewhere = bound
    bf, f32 = torch.bfloat16, torch.float32
    z = lambda *k, dt=bf: torch.zeros(*k, dtype=dt)  # noqa: E731
    L = hl.HSSAdapters(z(3, 6, 2), z(3, 2, 5))
    X, G, Y, ids = z(4, 5), z(4, 6), z(4, 6), torch.zeros(4, dtype=torch.int32)
    hl.hss_adapters_apply(L, X, ids), hl.hss_adapters_apply(L, X, ids, base=Y, Y=Y)
    hl.hss_adapters_grad(L, X, G, ids)
    hl.hss_adapters_grad(L, X, G, ids, base=X, out={"dU": z(3, 6, 2, dt=f32)})
    assert calls == ["hss_adapters_apply"] * 2 + ["hss_adapters_grad"] * 2
    bad_x = [z(4, 6), z(5, 5), X.float(), z(4, 10)[:, ::2], X[0], elsewhere(X)]
    bad_ids = [ids.long(), ids[:3], torch.zeros(8, dtype=torch.int32)[::2], elsewhere(ids), ids.view(4, 1)]
    bad_y = [z(4, 5), Y.float(), z(6, 4).t(), elsewhere(Y), z(3, 6)]
    bad_ws = [elsewhere(torch.zeros(1 << 16, dtype=torch.uint8)), torch.zeros(1 << 17, dtype=torch.uint8)[::2]]
    other = elsewhere(z(3, 6, 2))
    far = hl.HSSAdapters(other, elsewhere(z(3, 2, 5)))
    tries = [lambda x=x: hl.hss_adapters_apply(L, x, ids) for x in bad_x[:5]]
    tries += [lambda x=x: hl.hss_adapters_grad(L, x, G, ids) for x in bad_x[:5]]
    tries += [lambda i=i: hl.hss_adapters_apply(L, X, i) for i in bad_ids]
    tries += [lambda i=i: hl.hss_adapters_grad(L, X, G, i) for i in bad_ids]
    tries += [lambda y=y: hl.hss_adapters_apply(L, X, ids, Y=y) for y in bad_y]
    tries += [lambda y=y: hl.hss_adapters_apply(L, X, ids, base=y, Y=y) for y in bad_y]
    tries += [lambda y=y: hl.hss_adapters_grad(L, X, y, ids) for y in bad_y]
    tries += [lambda x=x: hl.hss_adapters_grad(L, X, G, ids, base=x) for x in bad_x]
    tries += [lambda w=w: hl.hss_adapters_apply(L, X, ids, ws=w) for w in bad_ws]
    tries += [lambda w=w: hl.hss_adapters_grad(L, X, G, ids, ws=w) for w in bad_ws]
    tries += [lambda o=o: hl.hss_adapters_grad(L, X, G, ids, out=o)
              for o in ({"dY": Y}, {"dX": Y}, {"dU": z(3, 6, 2)}, {"dU": z(6, 3, 2, dt=f32).transpose(0, 1)},
                        {"dVt": z(3, 2, 6, dt=f32)}, {"dVt": elsewhere(z(3, 2, 5, dt=f32))})]
    tries += [lambda: hl.hss_adapters_apply(far, X, ids), lambda: hl.hss_adapters_grad(far, X, G, ids)]
    for k, call in enumerate(tries):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(k)
    assert len(calls) == 4


def test_calls_refuse_cpu_tensors(hl):
    import torch
    bf = torch.bfloat16
    L = hl.HSSAdapters(torch.zeros(1, 6, 2, dtype=bf), torch.zeros(1, 2, 5, dtype=bf))
    X, G, ids = torch.zeros(4, 5, dtype=bf), torch.zeros(4, 6, dtype=bf), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: hl.hss_adapters_apply(L, X, ids), lambda: hl.hss_adapters_grad(L, X, G, ids)):
        with pytest.raises(ValueError):
            call()
