"""The AdamW step without a GPU: the oracle pinned by hand values, by fp64
arithmetic of its definition and by counts of its random rounding, and the
library's refusals (every call below fails its argument checks before any
device work)."""
import ctypes

import numpy as np
import pytest

import oracle as O

FAKE = 1 << 24  # never dereferenced


@pytest.fixture(scope="module")
def hl():
    import sparse_rank_linear_hss_amd as h
    return h


# ---------------------------------------------------------------------------
# The oracle
# ---------------------------------------------------------------------------

def test_first_step_by_hand():
    """From zeros, the bias corrections undo the averages: p loses lr wd p, then
    lr times the gradient's sign (eps small)."""
    p, m, v = O.adamw([1.0, -2.0, 0.5], [0.1, -3.0, 0.0], np.zeros(3), np.zeros(3), lr=0.01, step=1, eps=1e-12,
                      weight_decay=0.1)
    assert np.allclose(m, [0.01, -0.3, 0.0]) and np.allclose(v, [1e-5, 9e-3, 0.0])
    assert np.allclose(p, [1 - 0.001 - 0.01, -2 + 0.002 + 0.01, 0.5 - 0.0005], atol=1e-9)


def test_closed_form_of_the_averages():
    """t steps of one gradient: m = (1 - b1^t) g, v = (1 - b2^t) g^2, and the
    corrected step is lr whatever t is."""
    p, m, v = np.array([3.0]), np.zeros(1), np.zeros(1)
    for t in range(1, 40):
        q, m, v = O.adamw(p, [0.5], m, v, lr=1e-3, step=t, eps=0.0, weight_decay=0.0, grad_scale=0.5)
        assert np.allclose(m, (1 - 0.9 ** t) * 0.25) and np.allclose(v, (1 - 0.999 ** t) * 0.0625)
        assert np.allclose(p - q, 1e-3)
        p = q


def test_codes_are_e4m3():
    torch = pytest.importorskip("torch")
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.moment8_decode(codes, np.ones(1)), want)


def test_codes_keep_what_they_hold():
    """A value that a code holds is kept, whatever the random number is."""
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    x = O.moment8_decode(codes, np.ones(1))
    for u in (0, 1, 40000, 65535):
        got = O.moment8_encode(x, np.ones(1), np.full(len(x), u, np.uint32), 0)
        assert np.array_equal(got & 127, codes & 127) and np.array_equal(O.moment8_decode(got, np.ones(1)), x)


def test_rounding_takes_the_upper_code_in_proportion():
    """Between 16 (code 0x58) and 18 (0x59), and between 0 and 2^-9: the upper
    one where share + u / 2^16 >= 1, for floor(2^16 share) of the random numbers."""
    u = np.arange(65536, dtype=np.uint32)
    for low, step, c in ((16.0, 2.0, 0x58), (0.0, 2.0 ** -9, 0), (208.0, 16.0, 0x75)):
        for share in (0.0, 0.25, 0.7, 1 - 2.0 ** -16):
            x = np.full(65536, low + step * share)
            got = O.moment8_encode(x, np.ones(256), u, 0)
            assert set(got) <= {c, c + 1} and np.count_nonzero(got == c + 1) == int(65536 * share)


def test_scales_and_the_smallest_code():
    x = np.zeros(600)
    x[3], x[300], x[599] = -44.8, 1e-40, 2.0 ** -30
    x[4] = 1e-20
    s = O.moment8_scales(x)
    assert s.tolist() == [44.8 * (1 / 448), 0.0, 2.0 ** -30 * (1 / 448)]
    c = O.moment8_encode(x, s, np.zeros(600, np.uint32), 1)
    assert c[3] == 0x80 | 126 and c[4] == 1 and c[300] == 0 and c[599] == 126 and np.count_nonzero(c) == 3
    x[3] = np.inf
    assert not np.isfinite(O.moment8_scales(x)[0])
    assert np.all(np.isnan(O.moment8_decode(np.zeros(256, np.uint8), np.array([np.inf]))))


def test_hash_bits_are_even_and_apart():
    """Bits of the two halves, over positions and over steps: as many ones as
    zeros and no correlation, within five deviations."""
    n = 1 << 18
    h = [O.adamw_hash(np.arange(n), t) for t in (1, 2, 1000)]
    assert O.adamw_hash([0], 0)[0] == 0 and len(set(h[0].tolist())) == n     # a bijection of the position
    b = np.concatenate([((x[:, None] >> np.arange(32, dtype=np.uint32)) & 1) for x in h], axis=1).astype(np.float64) - 0.5
    assert np.all(np.abs(b.mean(axis=0)) < 5 * 0.5 / np.sqrt(n))
    c = (b.T @ b) / n * 4
    assert np.max(np.abs(c - np.eye(96))) < 5.5 / np.sqrt(n)
    assert np.max(np.abs((b[1:].T @ b[:-1]) / n * 4)) < 5.5 / np.sqrt(n)


# ---------------------------------------------------------------------------
# Refusals
# ---------------------------------------------------------------------------

def _call(hl, n=1, tensors=None, config=None, **kw):
    c = hl._lib.HssAdamwConfigStruct(bits=32, dtype=1, grad_dtype=0, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
                                     weight_decay=0.01, grad_scale=1.0, step=1)
    t, g = (hl._lib.HssAdamwTensorStruct * max(n, 1))(), (ctypes.c_void_p * max(n, 1))()
    for k in range(n):
        at = FAKE * (1 + 8 * (n - 1 - k))   # the last one, which kw changes, from FAKE on
        t[k].count, t[k].param, t[k].m, t[k].v = 1000, at, at + 2 * FAKE, at + 3 * FAKE
        g[k] = at + FAKE
        t[k].m_scale, t[k].v_scale = at + 5 * FAKE, at + 6 * FAKE
    for k, x in kw.items():
        if k == "grad":
            g[n - 1] = x
        elif k != "grads":
            setattr(c if hasattr(c, k) else t[n - 1], k, x)
    return hl._lib.lib.hss_adamw(ctypes.byref(c) if config is None else config, t if tensors is None else tensors,
                                 kw.get("grads", g), n, None)


def test_library_refuses(hl):
    INV = hl._lib.HSS_ERR_INVALID_ARG
    P = ctypes.POINTER
    assert _call(hl, config=P(hl._lib.HssAdamwConfigStruct)()) == INV
    assert _call(hl, tensors=P(hl._lib.HssAdamwTensorStruct)()) == INV
    assert _call(hl, n=-1) == INV
    nan, inf = float("nan"), float("inf")
    for bad in (dict(bits=16), dict(bits=0), dict(dtype=2), dict(grad_dtype=-1), dict(reserved=1), dict(lr=nan), dict(lr=inf),
                dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=nan), dict(eps=-1e-9), dict(eps=inf),
                dict(weight_decay=nan), dict(grad_scale=inf), dict(step=0), dict(step=-3), dict(step=2 ** 31),
                dict(count=-1), dict(count=2 ** 31), dict(param=None), dict(grads=None), dict(m=None), dict(v=None),
                dict(param=FAKE + 1), dict(grad=2 * FAKE + 2), dict(m=3 * FAKE + 1), dict(v=4 * FAKE + 2),
                dict(dtype=0, master=5 * FAKE), dict(master=5 * FAKE + 2), dict(master=2 * FAKE),
                dict(grad=FAKE), dict(m=FAKE + 1996), dict(v=3 * FAKE + 3996),
                dict(bits=8, m_scale=None), dict(bits=8, v_scale=None), dict(bits=8, m_scale=6 * FAKE + 2),
                dict(bits=8, v_scale=6 * FAKE), dict(bits=8, m_scale=4 * FAKE + 500)):
        assert _call(hl, **bad) == INV, bad
        if not any(hasattr(hl._lib.HssAdamwConfigStruct, k) for k in bad):
            assert _call(hl, n=3, **bad) == INV, bad                    # in a later tensor
    assert _call(hl, n=0) == hl._lib.HSS_OK
    assert _call(hl, count=0, param=None) == hl._lib.HSS_OK             # no element: nothing to do
    assert _call(hl, param=None, grad=None) == hl._lib.HSS_OK           # no gradient


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
        def hss_adamw(self, *a):
            calls.append(a)
            return 0

    monkeypatch.setattr(hl, "lib", Lib())
    monkeypatch.setattr(hl, "_current_device", lambda: -1)
    monkeypatch.setattr(hl, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(hl, "_index", lambda t: t.get_device())
    return calls, lambda t: t.as_subclass(Elsewhere)


def test_states_refuse_what_does_not_fit(hl, bound):
    import torch
    _, elsewhere = bound
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    ps = [torch.zeros(300, dtype=bf), torch.zeros(4, 5, dtype=bf)]
    s = hl.AdamWState(ps, bits=8, master=True)
    assert [t.numel() for t in s.m_scale] == [2, 1] and s.m[0].dtype == f8 and s.master[1].dtype == torch.float32
    again = hl.AdamWState(ps, bits=8, master=s.master, m=s.m, v=s.v, m_scale=s.m_scale, v_scale=s.v_scale)
    assert again.m[0] is s.m[0]
    z = lambda k, dt=torch.float32: torch.zeros(k, dtype=dt)  # noqa: E731
    for args, kw in (([[]], {}), ([ps], dict(bits=16)), ([[ps[0], z(3)]], {}), ([[z((6, 6), bf)[:, ::2]]], {}),
                     ([[ps[0], ps[0]]], {}), ([[ps[0], ps[0][10:]]], {}), ([[ps[0], elsewhere(ps[1])]], {}),
                     ([[z(4)]], dict(master=True)), ([ps], dict(master=[z(300)])), ([ps], dict(master=[z(300), z(21)])),
                     ([ps], dict(master=[z(300), z(20, bf)])), ([ps], dict(m=[z(300, f8), z(20, f8)])),
                     ([ps], dict(bits=8, m=[z(300), z(20)])), ([ps], dict(m=[z(300), z(40)[::2]])),
                     ([ps], dict(v=[z(300)])), ([ps], dict(m_scale=[z(2), z(1)])),
                     ([ps], dict(bits=8, m_scale=[z(1), z(1)])), ([ps], dict(bits=8, v_scale=[z(2), elsewhere(z(1))]))):
        with pytest.raises(ValueError):
            hl.AdamWState(*args, **kw)
    for dt in (torch.float16, torch.int32):
        with pytest.raises(TypeError):
            hl.AdamWState([torch.zeros(3, dtype=dt)])


def test_steps_refuse_what_does_not_fit(hl, bound):
    import torch
    calls, elsewhere = bound
    z = lambda k, dt=torch.float32: torch.zeros(k, dtype=dt)  # noqa: E731
    s = hl.AdamWState([z(300), z((4, 5))])
    hl.hss_adamw(s, [z(300), z(20)], 1e-3, 1)
    hl.hss_adamw(s, [None, z((4, 5), torch.bfloat16)], z(1), z(1, torch.int32), grad_scale=z(()))
    hl.hss_adamw(s, [None, None], 1e-3, 1)
    assert len(calls) == 3 and [list(c[2]) for c in calls][2] == [None, None] and calls[1][2][0] is None and calls[1][2][1]
    for grads, lr, step, kw in (([z(300)], 1e-3, 1, {}), ([z(300), z(21)], 1e-3, 1, {}), ([z(600)[::2], z(20)], 1e-3, 1, {}),
                                ([z(300), z(20, torch.bfloat16)], 1e-3, 1, {}), ([z(300), elsewhere(z(20))], 1e-3, 1, {}),
                                ([z(300), z(20)], z(2), 1, {}), ([z(300), z(20)], z(1, torch.float64), 1, {}),
                                ([z(300), z(20)], 1e-3, z(1, torch.int64), {}), ([z(300), z(20)], 1e-3, elsewhere(z(1, torch.int32)), {}),
                                ([z(300), z(20)], 1e-3, 1, dict(grad_scale=z(2)))):
        with pytest.raises(ValueError):
            hl.hss_adamw(s, grads, lr, step, **kw)
    with pytest.raises(TypeError):
        hl.hss_adamw(s, [z(300, torch.float16), z(20, torch.float16)], 1e-3, 1)
    assert len(calls) == 3


@pytest.mark.parametrize("step,seen", [(2 ** 64 + 1, 1 << 31), (2 ** 31, 1 << 31), (-2 ** 64 + 1, 0), (0, 0), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_a_step_out_of_range_does_not_wrap(hl, bound, step, seen):
    """The library refuses 0 and 2^31 (test_library_refuses)."""
    import torch
    calls, _ = bound
    s = hl.AdamWState([torch.zeros(3)])
    hl.hss_adamw(s, [torch.zeros(3)], 1e-3, step)
    assert len(calls) == 1 and s._config.step == seen


def test_cpu_tensors_are_refused(hl):
    import torch
    with pytest.raises(ValueError):
        hl.AdamWState([torch.zeros(3)])


_NO_DEVICE = """
import ctypes, sys
import torch
assert torch.cuda.device_count() == 0 and not torch.cuda.is_available()
import sparse_rank_linear_hss_amd as hl
live, left_out = int(sys.argv[1]), int(sys.argv[2])
n = live + left_out
c = hl._lib.HssAdamwConfigStruct(bits=32, dtype=0, grad_dtype=0, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
                                 weight_decay=0.01, grad_scale=1.0, step=1)
t, g = (hl._lib.HssAdamwTensorStruct * n)(), (ctypes.c_void_p * n)()
for k in range(n):
    at = (k + 1) << 24
    t[k].count, t[k].param, t[k].m, t[k].v = 8, at, at + 4096, at + 8192
    g[k] = at + 12288 if k < live else None
print("status", hl._lib.lib.hss_adamw(ctypes.byref(c), t, g, n, None))
"""


@pytest.mark.parametrize("live,left_out", [(1, 0), (48, 0), (48, 1), (96, 7), (50, 3), (0, 5)])
def test_a_launch_that_fails_is_reported(hl, live, left_out):
    """On no device every launch fails, and the call says so, also where nothing but tensors without
    gradients comes after the last full launch (of 48 tensors)."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _NO_DEVICE, str(live), str(left_out)], cwd=root, capture_output=True, text=True,
                       timeout=300, env=dict(os.environ, HIP_VISIBLE_DEVICES="-1"))
    want = hl._lib.HSS_ERR_HIP if live else hl._lib.HSS_OK
    assert r.stdout.split()[-2:] == ["status", str(want)], r.stdout + r.stderr


def test_scalars_off_their_grid_are_refused(hl):
    """The kernel reads a device scalar by its aligned word."""
    INV = hl._lib.HSS_ERR_INVALID_ARG
    for name in ("lr_dev", "step_dev", "grad_scale_dev"):
        for off in (1, 2, 3):
            assert _call(hl, **{name: 40 * FAKE + off}) == INV, (name, off)
            assert _call(hl, n=0, **{name: 40 * FAKE + off}) == INV, (name, off)
        assert _call(hl, n=0, **{name: 40 * FAKE + 4}) == hl._lib.HSS_OK


def test_a_step_refuses_parameters_with_other_memory(hl, bound):
    """The state holds the addresses that the step writes to: a parameter's memory may be someone else's
    by now.  Moments whose tensor was given other memory keep what the step writes to."""
    import gc
    import weakref

    import torch
    calls, _ = bound
    p, q = torch.nn.Parameter(torch.zeros(300)), torch.zeros(20)
    s = hl.AdamWState([p, q])
    hl.hss_adamw(s, [None, torch.zeros(20)], 1e-3, 1)
    held = p.data
    p.data = torch.ones(300)
    for grads in ([torch.zeros(300), None], [None, torch.zeros(20)], [None, None]):
        with pytest.raises(ValueError, match="memory"):
            hl.hss_adamw(s, grads, 1e-3, 1)
    p.data = held                                                       # the old memory again
    hl.hss_adamw(s, [torch.zeros(300), None], 1e-3, 1)
    q.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="memory"):
        hl.hss_adamw(s, [torch.zeros(300), None], 1e-3, 1)
    assert len(calls) == 2
    with pytest.raises(TypeError):
        s.m[0] = torch.zeros(300)
    own = np.ones(64, np.float32)
    alive = weakref.ref(own)
    m = torch.from_numpy(own)
    s = hl.AdamWState([torch.zeros(64)], m=[m])
    m.data = torch.zeros(64)
    del own
    gc.collect()
    assert alive() is not None


def test_a_step_is_a_change_in_place_for_autograd(hl, bound):
    """A backward pass that has saved a parameter's old values is refused after the step, as after any
    change in place; a parameter that the step leaves alone stays usable."""
    import torch
    w, o = torch.nn.Parameter(torch.ones(8)), torch.nn.Parameter(torch.ones(8))
    x = torch.ones(8, requires_grad=True)
    s = hl.AdamWState([w, o])
    y, z = (x * w).sum(), (x * o).sum()
    hl.hss_adamw(s, [torch.zeros(8), None], 1e-3, 1)
    z.backward()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        s = hl.AdamWState([torch.zeros(8)])
        hl.hss_adamw(s, [torch.zeros(8)], 1e-3, 1)
    with pytest.raises(ValueError):                                     # a refused step changes nothing
        hl.hss_adamw(hl.AdamWState([w]), [torch.zeros(9)], 1e-3, 1)
    (x * w).sum().backward()
