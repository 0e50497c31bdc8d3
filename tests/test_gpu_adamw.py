"""GPU parity of the AdamW step against the CPU oracle: bit for bit against its
operations in fp32, each rounded by itself (the step's definition), and within
derived bounds of its formula in fp64.

Bounds of the second, u = 2^-24 (half a step of fp32), N the sums of magnitudes:
    m: the scaled gradient, the two constants, two products, the sum   5 u N_m
    v: the same with the square, all of one sign                       8 u v
    sqrt(v) / .. + eps: half of v's, the root, the constants, two      10 u
    p: p (1 - lr wd): constant and product 2 u |p|; the quotient with m's
       5 u N_m over the denominator, 10 u, its constant and two more roundings;
       the difference u: in all 3 u |p| + size (5 u N_m + 14 u |m|) / denominator
    bf16 parameters: half a step more, 2^-8 of the value."""
import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24
HYPER = dict(beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


@pytest.fixture(scope="module")
def H():
    import sparse_rank_linear_hss_amd as h
    return h


def _bf16(x):
    import torch
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().float().numpy()


def _offset(a, dtype, shift):
    """a on the GPU, `shift` elements past a 16-byte boundary, with guards of 9
    elements around it; returns (view, guards intact?)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    raw = dtype == torch.float8_e4m3fn
    buf = torch.full((len(a) + shift + 9,), 77, dtype=torch.uint8 if raw else dtype, device="cuda")
    buf[shift:shift + len(a)] = t.cuda().to(buf.dtype)
    view = buf[shift:shift + len(a)]
    return (view.view(dtype) if raw else view), \
        lambda: bool((buf[:shift] == 77).all()) and bool((buf[shift + len(a):] == 77).all())


class Case:
    """Tensors of the given sizes with their moments in numpy, and the same on the GPU."""

    def __init__(self, H, sizes, p, g, bits, seed, shift=0, fresh=False, loud=1.0):
        import torch
        rng = np.random.default_rng(seed)
        self.p, self.g, self.bits = p, g, bits
        pdt = torch.float32 if p == "f32" else torch.bfloat16
        gdt = torch.float32 if g == "f32" else torch.bfloat16
        f8 = torch.float8_e4m3fn
        self.host, self.guards = [], []
        dev = {k: [] for k in ("param", "master", "grad", "m", "v", "m_scale", "v_scale")}

        def put(name, a, dt):
            t, ok = _offset(a, dt, shift)
            dev[name].append(t)
            self.guards.append(ok)

        for n in sizes:
            h = {}
            w = (0.05 * rng.standard_normal(n)).astype(np.float32)
            big = loud * 1e-3 * np.exp(rng.standard_normal(n))
            grad = (big * rng.standard_normal(n)).astype(np.float32)
            m = (0.3 * big * rng.standard_normal(n)).astype(np.float32)
            root = (big * (0.01 + rng.random(n))).astype(np.float32)
            if fresh:
                m[:], root[:] = 0, 0
            h["w"] = w if p != "bf16" else _bf16(w)
            h["g"] = grad if g == "f32" else _bf16(grad)
            put("grad", h["g"], gdt)
            put("param", w if p == "f32" else _bf16(w), pdt)
            if p == "bf16+f32":
                put("master", w, torch.float32)
            if bits == 32:
                h["m"], h["v"] = m, root * root
                put("m", m, torch.float32), put("v", h["v"], torch.float32)
            else:
                zero = np.zeros(n, np.uint32)
                for name, x in (("m", m), ("v", root)):
                    s = O.moment8_scales(x)
                    c = O.moment8_encode(x, s, zero, 0)
                    put(name, c, f8), put(name + "_scale", s.astype(np.float32), torch.float32)
                    h[name] = O.moment8_decode(c, s)
                    h[name] = h[name].astype(np.float32)                # the product rounds, as in the step
                h["v"] = h["v"] * h["v"]
            self.host.append(h)
        kw = {k: dev[k] for k in ("m", "v", "master", "m_scale", "v_scale") if dev[k]}
        self.dev = dev
        self.state = H.AdamWState(dev["param"], bits=bits, **kw)

    def check(self, step, lr=1e-3, grad_scale=1.0, skip=()):
        """What the device holds against one step from the host's."""
        import torch
        at = 0
        for k, h in enumerate(self.host):
            n = len(h["w"])
            if k in skip or n == 0:
                continue
            f32 = O.adamw(h["w"], h["g"], h["m"], h["v"], lr, step, grad_scale=grad_scale, dtype=np.float32, **HYPER)
            f64 = O.adamw(h["w"], h["g"], h["m"], h["v"], lr, step, grad_scale=grad_scale, **HYPER)
            holder = self.dev["master"][k] if self.p == "bf16+f32" else self.dev["param"][k]
            got = holder.float().cpu().numpy()
            want = f32[0] if self.p != "bf16" else _bf16(f32[0])
            assert np.array_equal(got, want)
            if self.p == "bf16+f32":
                assert np.array_equal(self.dev["param"][k].float().cpu().numpy(), _bf16(f32[0]))
            x = np.abs(h["g"].astype(np.float64) * grad_scale)
            n_m = 0.9 * np.abs(h["m"]) + 0.1 * x
            size, root = lr / (1 - 0.9 ** step), 1 / np.sqrt(1 - 0.999 ** step)
            den = np.sqrt(f64[2]) * root + 1e-8
            tol = 3 * U24 * np.abs(h["w"]) + size * U24 * (5 * n_m + 14 * np.abs(f64[1])) / den + 2.0 ** -149
            tol = tol + (2.0 ** -8 * np.abs(f64[0]) if self.p == "bf16" else 0)
            assert np.all(np.abs(got - f64[0]) <= tol * (1 + 2.0 ** -8))
            if self.bits == 32:
                m, v = self.dev["m"][k].cpu().numpy(), self.dev["v"][k].cpu().numpy()
                assert np.array_equal(m, f32[1]) and np.array_equal(v, f32[2])
                assert np.all(np.abs(m - f64[1]) <= 5 * U24 * n_m + 2.0 ** -148)
                assert np.all(np.abs(v - f64[2]) <= 8 * U24 * f64[2] + 2.0 ** -148)
            else:
                u = O.adamw_hash(at + np.arange(n), step)
                for name, y, rnd, least in (("m", f32[1], u & 0xffff, 0), ("v", np.sqrt(f32[2]), u >> 16, 1)):
                    s = O.moment8_scales(y)
                    assert np.array_equal(self.dev[name + "_scale"][k].cpu().numpy(), s)
                    assert np.array_equal(self.dev[name][k].view(torch.uint8).cpu().numpy(),
                                          O.moment8_encode(y, s, rnd, least))
            at += -(-n // O.ADAMW_BLOCK) * O.ADAMW_BLOCK
        assert all(ok() for ok in self.guards)


SIZES = [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 5003]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("g", ["f32", "bf16"])
@pytest.mark.parametrize("p", ["f32", "bf16", "bf16+f32"])
@pytest.mark.parametrize("shift", [0, 1])
def test_step(H, p, g, bits, shift):
    """Every type, ragged sizes, arrays on and off the 16-byte grid."""
    c = Case(H, SIZES, p, g, bits, seed=bits + shift, shift=shift)
    H.hss_adamw(c.state, c.dev["grad"], lr=1e-3, step=11)
    c.check(11)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("step", [1, 2, 1000, 2 ** 31 - 1])
def test_first_and_late_steps(H, bits, step):
    c = Case(H, [700, 3], "bf16+f32", "f32", bits, seed=5, fresh=step == 1)
    H.hss_adamw(c.state, c.dev["grad"], lr=1e-3, step=step)
    c.check(step)


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_launch_takes(H, bits):
    """130 tensors, some without elements, some without a gradient; the
    positions of the random numbers go on over the launches."""
    sizes = [(37 * k) % 700 for k in range(130)]
    sizes[5] = sizes[129] = 0
    c = Case(H, sizes, "f32", "f32", bits, seed=6)
    H.hss_adamw(c.state, c.dev["grad"], lr=1e-3, step=4)
    c.check(4)
    c = Case(H, sizes, "bf16", "f32", bits, seed=7)
    skip = {0, 3, 60, 61}
    before = [[t.clone() for t in c.dev[k]] for k in ("param", "m", "v")]
    H.hss_adamw(c.state, [None if k in skip else t for k, t in enumerate(c.dev["grad"])], lr=1e-3, step=4)
    c.check(4, skip=skip)
    for kept, now in zip(before, (c.dev["param"], c.dev["m"], c.dev["v"])):
        assert all(kept[k].float().equal(now[k].float()) for k in skip)


@pytest.mark.parametrize("bits", [32, 8])
def test_scalars_on_the_device(H, bits):
    """lr, step and grad_scale read from the GPU give the bits of the numbers."""
    import torch
    lr = float(np.float32(3e-4))
    dev = [torch.tensor([lr], device="cuda"), torch.tensor([9], dtype=torch.int32, device="cuda"),
           torch.tensor([0.25], device="cuda")]
    c = Case(H, SIZES, "bf16+f32", "bf16", bits, seed=8)
    H.hss_adamw(c.state, c.dev["grad"], lr=dev[0], step=dev[1], grad_scale=dev[2])
    c.check(9, lr=lr, grad_scale=0.25)
    c = Case(H, SIZES, "f32", "f32", bits, seed=8)
    H.hss_adamw(c.state, c.dev["grad"], lr=lr, step=dev[1], grad_scale=0.25)
    c.check(9, lr=lr, grad_scale=0.25)
    c = Case(H, SIZES, "f32", "f32", bits, seed=8)
    H.hss_adamw(c.state, c.dev["grad"], lr=lr, step=9, grad_scale=dev[2])
    c.check(9, lr=lr, grad_scale=0.25)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_follows_its_scalars(H, bits):
    """A step captured once and replayed, its step number advanced in the graph
    and its gradients and lr changed between replays, other work in between:
    the bits of the same steps run eagerly."""
    import torch
    runs = [Case(H, [5003, 64, 257], "bf16+f32", "f32", bits, seed=9) for _ in range(2)]
    lr, step = torch.tensor([1e-3], device="cuda"), torch.tensor([0], dtype=torch.int32, device="cuda")
    warm = Case(H, [64], "bf16+f32", "f32", bits, seed=1)
    H.hss_adamw(warm.state, warm.dev["grad"], lr=lr, step=step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        H.hss_adamw(runs[0].state, runs[0].dev["grad"], lr=lr, step=step)
    for t in range(1, 5):
        for r in runs:
            gen = torch.Generator(device="cuda").manual_seed(t)
            for g in r.dev["grad"]:
                g.copy_(1e-3 * torch.randn(g.shape, device="cuda", generator=gen))
        lr.fill_(1e-3 / t)
        graph.replay()
        H.hss_adamw(warm.state, warm.dev["grad"], lr=lr, step=t)
        H.hss_adamw(runs[1].state, runs[1].dev["grad"], lr=lr, step=t)
        torch.cuda.synchronize()
        assert step.item() == t
        for name in ("param", "master", "m", "v", "m_scale", "v_scale"):
            assert all(a.float().equal(b.float()) for a, b in zip(runs[0].dev[name], runs[1].dev[name])), (t, name)


def test_same_bits_on_another_stream_and_again(H):
    import torch
    a, b = (Case(H, SIZES, "bf16", "bf16", 8, seed=3) for _ in range(2))
    H.hss_adamw(a.state, a.dev["grad"], lr=1e-3, step=7)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        H.hss_adamw(b.state, b.dev["grad"], lr=1e-3, step=7)
    torch.cuda.synchronize()
    a.check(7), b.check(7)


@pytest.mark.parametrize("bits", [32, 8])
def test_non_finite_gradients_stay_where_they_are(H, bits):
    """One NaN and one infinity: their elements in fp32, their blocks of 256 in
    8 bits; every other value has the bits of a step without them."""
    import torch
    a, b = (Case(H, [1000, 600], "f32", "f32", bits, seed=4) for _ in range(2))
    for k, i, x in ((0, 300, float("nan")), (1, 599, float("inf"))):
        b.dev["grad"][k][i] = x
    for c in (a, b):
        H.hss_adamw(c.state, c.dev["grad"], lr=1e-3, step=3)
    for k, i, lo, hi in ((0, 300, 256, 512), (1, 599, 512, 600)):
        near = torch.zeros(len(a.host[k]["w"]), dtype=torch.bool, device="cuda")
        near[i] = True
        assert not torch.isfinite(b.dev["param"][k][i])
        assert torch.equal(a.dev["param"][k][~near], b.dev["param"][k][~near])
        if bits == 8:
            near[lo:hi] = True
            scale = [c.dev["m_scale"][k].repeat_interleave(256)[:len(near)] for c in (a, b)]
            value = [c.dev["m"][k].float() * s for c, s in zip((a, b), scale)]
            assert torch.equal(value[0][~near], value[1][~near]) and bool(value[1][near].isnan().all())
        else:
            assert torch.equal(a.dev["v"][k][~near], b.dev["v"][k][~near]) and not torch.isfinite(b.dev["v"][k][i])


def test_tiny_and_zero_blocks_of_8_bit_moments(H):
    """A block without gradients stays zero, one whose scale falls below 2^-100
    is kept as zeros, and no sqrt(v) above 0 beside a large one becomes 0."""
    import torch
    c = Case(H, [1024], "f32", "f32", 8, seed=2, fresh=True)
    g = c.dev["grad"][0]
    g[:256] = 0
    g[256:512] = 1e-29
    g[512:768] = 1e-18
    g[512] = 1.0
    c.host[0]["g"] = g.cpu().numpy()
    H.hss_adamw(c.state, c.dev["grad"], lr=1e-3, step=1)
    c.check(1)
    code = c.dev["v"][0].view(torch.uint8)
    assert not code[:512].any() and not c.dev["v_scale"][0][:2].any()
    assert bool((code[513:768] == 1).all()) and code[512] == 126


def test_slow_average_in_8_bits_moves_in_the_mean(H):
    """sqrt(v) a hundred steps after the gradients became eight times larger: a
    step of b2 changes it by less than half a code, so the nearest code would
    have stopped; the mean over 65,536 elements follows the fp64 average.  Its
    deviation: each step's rounding adds at most half a code (2^-4) of variance
    p (1 - p), p <= 0.26 the share of a code that a step moves; over 100 steps and
    65,536 elements that is below 0.0625 * sqrt(100 * 0.2 / 65536) = 0.0011 of the
    value, and five of them 0.0055.  The square of a noisy root is larger in the mean
    by the noise's own variance, at most 0.0625^2 * 100 * 0.2 / 2 = 0.039 of
    sqrt(v); together below 0.05."""
    import torch
    n = 65536
    p = torch.zeros(n, device="cuda")
    s = H.AdamWState([p], bits=8)
    g = torch.full((n,), 1.0, device="cuda")
    v = 0.0
    for t in range(1, 121):
        x = 1.0 if t <= 20 else 8.0
        g.fill_(x)
        H.hss_adamw(s, [g], lr=0.0, step=t)
        v = 0.999 * v + 0.001 * x * x
    root = (s.v[0].float() * s.v_scale[0].repeat_interleave(256)).double().mean().item()
    assert abs(root / v ** 0.5 - 1) < 0.05


def test_after_a_backward_pass(H):
    """Forward, backward and step of a compressed layer, the transposed layer
    written again: S's values, U and V^T are those of the oracle's step from the
    gradients that the backward pass returned, and the next forward uses them."""
    import torch

    import hss_synth as syn
    from _cases import to_dev
    m, n, r, b = 96, 160, 12, 33
    sp = H.hss_split(to_dev(syn.random_matrix(m, n, O.BF16, seed=1, kind="t3"), O.BF16), "csr", frac=(5, 100))
    U, V = syn.factors(m, n, r, O.BF16, 2)
    A = H.HSSMatrix.from_split(sp, U=to_dev(U, O.BF16), Vt=to_dev(np.ascontiguousarray(V.T), O.BF16))
    At = H.hss_transposed_layer(A)
    X = to_dev(syn.random_matrix(b, n, O.BF16, seed=3, kind="normal", scale=1.0), O.BF16)
    G = to_dev(syn.random_matrix(b, m, O.BF16, seed=4, kind="normal", scale=1.0), O.BF16)
    params = [A.values, A.U, A.Vt]
    state = H.AdamWState(params, bits=8, master=True)
    Y = H.hss_apply(A, X)
    for t in (1, 2):
        before = [w.clone() for w in state.master]
        held = [[x.float().clone() for x in state.m], [x.float().clone() for x in state.v],
                [x.clone() for x in state.m_scale], [x.clone() for x in state.v_scale]]
        g = H.hss_backward(A, X, G, At)
        grads = [g["dS"], g["dU"], g["dVt"]]
        H.hss_adamw(state, grads, lr=1e-2, step=t)
        H.hss_transposed_layer(A, out=At)
        for k, w in enumerate(params):
            k_of = len(w.view(-1))
            mm = (held[0][k] * held[2][k].repeat_interleave(256)[:k_of]).cpu().numpy()
            root = (held[1][k] * held[3][k].repeat_interleave(256)[:k_of]).cpu().numpy()
            want = O.adamw(before[k].cpu().numpy(), grads[k].reshape(-1).cpu().numpy(), mm, root * root, 1e-2, t,
                           dtype=np.float32, **HYPER)[0]
            assert np.array_equal(state.master[k].cpu().numpy(), want)
            assert np.array_equal(w.float().view(-1).cpu().numpy(), _bf16(want))
    fresh = H.hss_transposed_layer(A)
    assert torch.equal(At.U, fresh.U) and torch.equal(At.Vt, fresh.Vt) and torch.equal(At.values, fresh.values)
    assert not torch.equal(H.hss_apply(A, X), Y)


def test_a_million_elements_a_tensor(H):
    """A tensor of many passes of the grid beside a small one."""
    c = Case(H, [4_500_001, 5], "bf16+f32", "f32", 8, seed=12)
    H.hss_adamw(c.state, c.dev["grad"], lr=1e-3, step=100)
    c.check(100)


@pytest.mark.parametrize("on", ["lr", "lr and grad_scale", "lr and step"])
def test_a_rate_on_the_device_rounds_as_the_number(H, on):
    """The step's size lr / (1 - b1^t), in fp64 and rounded once, wherever lr is: the bits of the number
    at 1000 steps of several rates, from p = 0, where p = -size * quotient shows the size's last bit."""
    import torch
    rates = [float(np.float32(x)) for x in (1e-3, 3e-4, 1e-4, 0.7, 6.1e-6)]
    gen = torch.Generator(device="cuda").manual_seed(1)
    g = torch.randn(64, device="cuda", generator=gen)
    states = [H.AdamWState([torch.zeros(64, device="cuda")]) for _ in range(2)]
    lr = torch.zeros(1, device="cuda")
    scale = torch.full((1,), 0.5, device="cuda")
    steps = torch.arange(1, 1001, dtype=torch.int32, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    assert any(np.float32(x / np.float32(1 - 0.9 ** t)) != np.float32(x / (1 - 0.9 ** t)) for x in rates for t in range(1, 9))
    for x in rates:
        lr.fill_(x)
        for t in range(1, 1001):
            for s in states:
                s.params[0].zero_()
            H.hss_adamw(states[0], [g], lr=x, step=t, grad_scale=0.5)
            H.hss_adamw(states[1], [g], lr=lr, step=steps[t - 1] if "step" in on else t, grad_scale=scale if "grad" in on else 0.5)
            wrong += (states[0].params[0] != states[1].params[0]).sum()
    assert wrong.item() == 0


def test_small_codes_round_as_they_are_defined(H):
    """Values below the codes' smallest step, 2^-9 of a scale: the upper code only where share + u / 2^16 >=
    1, exactly.  At the elements whose random numbers are the largest, shares just below 1 - u / 2^16, by
    less than fp32 tells from 1 once the two are added."""
    import torch
    n, step = 1 << 18, 1
    h = O.adamw_hash(np.arange(n), step)
    g = np.full(n, 1e-6, np.float32)
    g[::256] = 1.0                                                       # the blocks' largest
    m1 = np.float32(1.0 - 0.9) * np.float32(1.0)
    scale = m1 * np.float32(1.0 / 448)
    u = (h & 0xffff).astype(np.int64)
    at = np.flatnonzero((u >= 65536 - 64) & (np.arange(n) % 256 != 0))
    share = (65536 - u[at]) / 65536.0 * (1 - 2.0 ** -16)
    g[at] = (share / 512 * float(scale) / float(np.float32(1.0 - 0.9))).astype(np.float32)
    m = np.float32(1.0 - 0.9) * g
    want = O.moment8_encode(m, O.moment8_scales(m), h & 0xffff, 0)
    a = np.abs(m) * (np.float32(1) / scale)
    summed = (a[at] * np.float32(512) + u[at].astype(np.float32) * np.float32(2.0 ** -16)).astype(np.int64)
    assert len(at) > 50 and not want[at].any() and np.count_nonzero(summed) > 50      # what a sum in fp32 would give
    s = H.AdamWState([torch.zeros(n, device="cuda")], bits=8)
    H.hss_adamw(s, [torch.from_numpy(g).cuda()], lr=1e-3, step=step)
    assert np.array_equal(s.m[0].view(torch.uint8).cpu().numpy(), want)
