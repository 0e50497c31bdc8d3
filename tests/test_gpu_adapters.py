"""GPU parity of the adapters against the CPU oracle.

Bounds.  u = 2^-24 (half a step of fp32), bf16's half step 2^-8 of the value.  A
sum of K products of bf16 values in fp32, in any order, is off by at most K u
times the sum of magnitudes; N: the formula with every value's magnitude.
    Y   T = X Vt^T (n terms), times scale (1), in two bf16 terms (2^-16), 2 r
        products with U and base (2 r + 1), rounded:
        2^-8 |Y| + ((n + 2 r + 3) u + 2^-16) N;   dX the same with m for n
    dU  T as before in three terms (2^-24), products with G over b rows in
        three terms:  (n + 3 b + 3) u N;          dVt the same with m for n
The products of two such errors are below 2^-8 of them: a factor 1.01."""
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


def _rand(shape, seed, scale):
    rng = np.random.default_rng(seed)
    flat = (scale * rng.standard_normal(int(np.prod(shape)))).astype(np.float32)
    import torch
    return torch.from_numpy(flat).bfloat16().view(torch.int16).numpy().view(np.uint16).reshape(shape)


def _ids(kind, b, count, seed):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full(b, count - 1)
    if kind == "each":
        return rng.permutation(np.arange(b) % count)
    if kind == "runs":
        return np.sort(rng.integers(0, count, b))
    if kind == "none":
        return np.full(b, -1)
    # some without an adapter, by every number that means none
    out = rng.integers(0, count, b)
    odd = rng.random(b) < 0.3
    out[odd] = rng.choice([-1, count, -2 ** 31, 2 ** 31 - 1, count + 64], b)[odd]
    return out


class Case:
    def __init__(self, H, m, n, r, b, count, kind, seed=1, scaled=True, based=True, shift=0):
        import torch
        self.H, self.m, self.n, self.r, self.b, self.count = H, m, n, r, b, count
        raw = {"U": _rand((count, m, r), seed, 0.1), "Vt": _rand((count, r, n), seed + 1, 0.1), "X": _rand((b, n), seed + 2, 1.0),
               "G": _rand((b, m), seed + 3, 0.1), "base": _rand((b, m), seed + 4, 1.0), "dbase": _rand((b, n), seed + 5, 0.1)}
        self.f = {k: O.widen(v, BF) for k, v in raw.items()}
        self.d = {}
        for k, v in raw.items():  # `shift` elements past a 16-byte boundary
            buf = torch.zeros(v.size + shift + 8, dtype=torch.bfloat16, device="cuda")
            self.d[k] = buf[shift:shift + v.size].view(v.shape)
            self.d[k].copy_(to_dev(v, BF))
        self.ids = _ids(kind, b, count, seed)
        self.ids_d = torch.from_numpy(self.ids.astype(np.int32)).cuda()
        self.scale = np.ones(count, np.float32)
        scale_d = None
        if scaled:
            self.scale = np.random.default_rng(seed).uniform(-2, 2, count).astype(np.float32)
            scale_d = torch.from_numpy(self.scale).cuda()
        self.based = based
        self.L = H.HSSAdapters(self.d["U"], self.d["Vt"], scale_d)

    def magnitudes(self):
        return {k: np.abs(v) for k, v in self.f.items()}, np.abs(self.scale)

    def apply_bound(self):
        f, (a, s) = self.f, self.magnitudes()
        base, abase = (f["base"], a["base"]) if self.based else (None, None)
        Y = O.adapters_apply(f["U"], f["Vt"], self.scale.astype(np.float64), f["X"], self.ids, base)
        N = O.adapters_apply(a["U"], a["Vt"], s, a["X"], self.ids, abase)
        return Y, (2.0 ** -8 * np.abs(Y) + ((self.n + 2 * self.r + 3) * U24 + 2.0 ** -16) * N) * 1.01

    def grad_bounds(self):
        f, (a, s) = self.f, self.magnitudes()
        base, abase = (f["dbase"], a["dbase"]) if self.based else (None, None)
        want = O.adapters_grad(f["U"], f["Vt"], self.scale.astype(np.float64), f["X"], f["G"], self.ids, base)
        N = O.adapters_grad(a["U"], a["Vt"], s, a["X"], a["G"], self.ids, abase)
        tol = [2.0 ** -8 * np.abs(want[0]) + ((self.m + 2 * self.r + 3) * U24 + 2.0 ** -16) * N[0],
               (self.n + 3 * self.b + 3) * U24 * N[1], (self.m + 3 * self.b + 3) * U24 * N[2]]
        return dict(zip(("dX", "dU", "dVt"), want)), dict(zip(("dX", "dU", "dVt"), (t * 1.01 for t in tol)))

    def apply(self, **kw):
        return self.H.hss_adapters_apply(self.L, self.d["X"], self.ids_d, base=self.d["base"] if self.based else None, **kw)

    def grad(self, **kw):
        return self.H.hss_adapters_grad(self.L, self.d["X"], self.d["G"], self.ids_d,
                                        base=self.d["dbase"] if self.based else None, **kw)

    def check_apply(self, Y):
        want, tol = self.apply_bound()
        got = Y.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / np.maximum(tol, 1e-300)))

    def check_grad(self, g, keys=("dX", "dU", "dVt")):
        want, tol = self.grad_bounds()
        for k in keys:
            err = np.abs(g[k].double().cpu().numpy() - want[k])
            assert np.all(err <= tol[k]), (k, float(np.max(err / np.maximum(tol[k], 1e-300))))


def _nan_ws(size):
    import torch
    return torch.full((size,), 255, dtype=torch.uint8, device="cuda")   # NaN as floats: what is not written shows


SHAPES = [(96, 64, 8), (1, 1, 1), (3, 7, 2), (257, 255, 15), (64, 1000, 17), (1000, 33, 32), (130, 514, 33), (300, 520, 64),
          (200, 300, 65), (65, 129, 130), (513, 2049, 16)]


@pytest.mark.parametrize("m,n,r", SHAPES)
@pytest.mark.parametrize("b,count,kind", [(1, 1, "one"), (2, 3, "mixed"), (17, 5, "mixed"), (64, 64, "each"), (40, 1, "one"),
                                          (65, 4, "runs"), (127, 9, "mixed"), (300, 3, "each")])
def test_apply_and_gradients(H, m, n, r, b, count, kind):
    c = Case(H, m, n, r, b, count, kind, seed=m + n + r + b)
    c.check_apply(c.apply(ws=_nan_ws(H.hss_adapters_workspace_size(c.L, b))))
    c.check_grad(c.grad(ws=_nan_ws(H.hss_adapters_grad_workspace_size(c.L, b))))


@pytest.mark.parametrize("b", [1, 15, 16, 31, 32, 33, 63, 64, 65, 66, 96, 97, 129, 1000, 2047, 2048])
@pytest.mark.parametrize("kind,count", [("one", 1), ("mixed", 7), ("runs", 40)])
def test_batches(H, b, kind, count):
    """Tiles of every fill, on both sides of the batch where their size changes."""
    c = Case(H, 80, 144, 24, b, count, kind, seed=b)
    c.check_apply(c.apply())
    c.check_grad(c.grad())


@pytest.mark.parametrize("b", [1, 50, 70, 2048])
def test_rows_without_an_adapter(H, b):
    """All of them: the outputs are base, or zeros, and the gradients zeros."""
    import torch
    for based in (True, False):
        c = Case(H, 100, 70, 9, b, 3, "none", based=based)
        Y, g = c.apply(), c.grad()
        assert torch.equal(Y, c.d["base"] if based else torch.zeros_like(Y))
        assert torch.equal(g["dX"], c.d["dbase"] if based else torch.zeros_like(g["dX"]))
        assert not g["dU"].any() and not g["dVt"].any()


@pytest.mark.parametrize("count,b", [(4096, 30), (4096, 2000), (1000, 65), (257, 300), (255, 300)])
def test_large_banks(H, count, b):
    c = Case(H, 24, 40, 3, b, count, "mixed", seed=count)
    c.check_apply(c.apply())
    c.check_grad(c.grad())


@pytest.mark.parametrize("m,n,r", [(90, 70, 257), (40, 600, 300), (530, 100, 513)])
@pytest.mark.parametrize("b,count,kind", [(1, 1, "one"), (30, 4, "mixed"), (100, 3, "mixed")])
def test_large_ranks(H, m, n, r, b, count, kind):
    """More of them than the forward keeps of T at a time."""
    c = Case(H, m, n, r, b, count, kind, seed=r + b)
    c.check_apply(c.apply(ws=_nan_ws(H.hss_adapters_workspace_size(c.L, b))))
    c.check_grad(c.grad(ws=_nan_ws(H.hss_adapters_grad_workspace_size(c.L, b))))


@pytest.mark.parametrize("m,n,r,count", [(300, 520, 41, 40), (300, 520, 100, 20), (255, 1025, 64, 40), (3, 257, 33, 64),
                                         (258, 2, 200, 20), (1000, 511, 48, 33)])
@pytest.mark.parametrize("b,kind", [(65, "mixed"), (300, "runs"), (515, "one")])
def test_gradients_of_many_columns_in_all(H, m, n, r, count, b, kind):
    """Blocks of 256 columns that share the terms (count ceil(r / 64) (ceil(m / 256) +
    ceil(n / 256)) >= 96), at ends of rows and ranks, with outputs left out."""
    import torch
    c = Case(H, m, n, r, b, count, kind, seed=r + b, shift=b % 2)
    full = c.grad(ws=_nan_ws(H.hss_adapters_grad_workspace_size(c.L, b)))
    c.check_grad(full)
    for keys in (("dU",), ("dVt",), ("dX", "dVt")):
        got = c.grad(**{k: k in keys for k in ("dX", "dU", "dVt")})
        assert all(torch.equal(got[k], full[k]) for k in keys)


@pytest.mark.parametrize("m,n,r,b,count,kind", [
    (1501, 2777, 41, 201, 5, "mixed"), (1300, 1100, 64, 2000, 4, "one"), (1300, 1101, 20, 1000, 5, "mixed"),
    (2049, 2100, 9, 2048, 2, "runs"), (4100, 4099, 30, 300, 1, "one"), (4099, 4100, 1, 64, 1, "mixed")])
def test_gradients_of_blocks_whose_waves_share_the_rows(H, m, n, r, b, count, kind):
    """Fewer columns in all than above, more than are split 32 a block ((m + n) count ceil(r / 64) >= 8192)."""
    c = Case(H, m, n, r, b, count, kind, seed=r + b)
    c.check_apply(c.apply(ws=_nan_ws(H.hss_adapters_workspace_size(c.L, b))))
    c.check_grad(c.grad(ws=_nan_ws(H.hss_adapters_grad_workspace_size(c.L, b))))


@pytest.mark.parametrize("b,r", [(30, 16), (30, 70), (300, 40)])
def test_two_streams_at_once(H, b, r):
    """One bank from two streams, each with outputs and a workspace of its own, one call after another."""
    import torch
    cases = [Case(H, 500, 700, r, b, 5, "mixed", seed=1)]
    cases.append(Case(H, 500, 700, r, b, 5, "each", seed=2))
    cases[1].L, cases[1].scale = cases[0].L, cases[0].scale
    want = [[c.apply(), *c.grad().values()] for c in cases]
    got = [[torch.empty_like(t) for t in w] for w in want]
    ws = [(H.adapters_workspace(c.L, b, "cuda"), H.adapters_grad_workspace(c.L, b, "cuda")) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(10):
        for g in got:
            for t in g:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            for c, g, w, s in zip(cases, got, ws, streams):
                with torch.cuda.stream(s):
                    c.apply(Y=g[0], ws=w[0])
                    c.grad(out=dict(zip(("dX", "dU", "dVt"), g[1:])), ws=w[1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, e) for g, w in zip(got, want) for a, e in zip(g, w))


def test_the_largest_bank(H):
    """4096 adapters of 524287 x 64, r = 1: 2^31 - 4096 values of U, 4 rows, more
    gradient blocks than one row of a grid takes.  The rows' adapters against the
    formula, all others' gradients zeros."""
    import torch
    count, m, n = 4096, 524287, 64
    ids = np.array([4095, 0, 4095, 2048])
    rng = np.random.default_rng(0)
    used = sorted(set(ids.tolist()))
    U = torch.zeros(count, m, 1, dtype=torch.bfloat16, device="cuda")
    Vt = torch.zeros(count, 1, n, dtype=torch.bfloat16, device="cuda")
    f = {}
    for l in used:
        u, v = _rand((m, 1), l + 1, 0.1), _rand((1, n), l + 2, 0.1)
        U[l], Vt[l] = to_dev(u, BF), to_dev(v, BF)
        f[l] = (O.widen(u, BF), O.widen(v, BF))
    X, G = _rand((4, n), 5, 1.0), _rand((4, m), 6, 0.1)
    L = H.HSSAdapters(U, Vt)
    Xd, Gd = to_dev(X, BF), to_dev(G, BF)
    ids_d = torch.from_numpy(ids.astype(np.int32)).cuda()
    X, G = O.widen(X, BF), O.widen(G, BF)
    at = {l: k for k, l in enumerate(used)}
    args = [np.stack([f[l][k] for l in used]) for k in (0, 1)] + [np.ones(len(used))]
    small = np.array([at[l] for l in ids])
    absolute = [np.abs(a) for a in args]
    got = H.hss_adapters_apply(L, Xd, ids_d).double().cpu().numpy()
    want, N = O.adapters_apply(*args, X, small), O.adapters_apply(*absolute, np.abs(X), small)
    assert np.all(np.abs(got - want) <= 1.01 * (2.0 ** -8 * np.abs(want) + ((n + 5) * U24 + 2.0 ** -16) * N))
    out = {"dU": torch.full((count, m, 1), float("nan"), device="cuda"), "dVt": torch.full((count, 1, n), float("nan"), device="cuda"),
           "dX": torch.empty_like(Xd)}
    H.hss_adapters_grad(L, Xd, Gd, ids_d, out=out)
    want, N = O.adapters_grad(*args, X, G, small), O.adapters_grad(*absolute, np.abs(X), np.abs(G), small)
    tol = [2.0 ** -8 * np.abs(want[0]) + ((m + 5) * U24 + 2.0 ** -16) * N[0], (n + 15) * U24 * N[1], (m + 15) * U24 * N[2]]
    for k, got in enumerate((out["dX"], out["dU"][used], out["dVt"][used])):
        assert np.all(np.abs(got.double().cpu().numpy() - want[k]) <= 1.01 * tol[k])
    out["dU"][used], out["dVt"][used] = 0, 0
    for k in ("dU", "dVt"):
        assert all(not part.any() for part in out[k].split(256))     # (a NaN counts)


@pytest.mark.parametrize("m,n,r,b,count", [(96, 64, 8, 5, 2), (130, 514, 33, 70, 3), (1000, 1000, 64, 100, 2)])
def test_arrays_off_the_16_byte_grid(H, m, n, r, b, count):
    for shift in (1, 3, 4):
        c = Case(H, m, n, r, b, count, "mixed", shift=shift)
        c.check_apply(c.apply())
        c.check_grad(c.grad())


@pytest.mark.parametrize("b", [3, 64, 65, 200])
def test_in_place_without_base_and_without_scale(H, b):
    import torch
    c = Case(H, 136, 200, 16, b, 4, "mixed")
    Y = c.apply()
    again = c.d["base"].clone()
    out = H.hss_adapters_apply(c.L, c.d["X"], c.ids_d, base=again, Y=again)
    assert out is again and torch.equal(again, Y)
    g = c.grad()
    again = c.d["dbase"].clone()
    out = H.hss_adapters_grad(c.L, c.d["X"], c.d["G"], c.ids_d, base=again, out={"dX": again})
    assert list(out) == ["dX"] and torch.equal(again, g["dX"])
    c = Case(H, 136, 200, 16, b, 4, "mixed", scaled=False, based=False)
    c.check_apply(c.apply())
    c.check_grad(c.grad())


@pytest.mark.parametrize("b", [9, 130])
def test_outputs_left_out_and_surroundings_left_alone(H, b):
    """Each output by itself has the bits of all together; nothing around the
    outputs is written."""
    import torch
    c = Case(H, 130, 70, 20, b, 3, "mixed")
    full = c.grad()
    for keys in (("dX",), ("dU",), ("dVt",), ("dU", "dVt"), ("dX", "dU")):
        got = c.grad(**{k: k in keys for k in ("dX", "dU", "dVt")})
        assert set(got) == set(keys) and all(torch.equal(got[k], full[k]) for k in keys)
    assert c.grad(dX=False, dU=False, dVt=False) == {}
    outs, guards = {}, []
    for k, t in [("Y", c.apply())] + list(full.items()):
        buf = torch.full((t.numel() + 77,), 123.0, dtype=t.dtype, device="cuda")
        outs[k] = buf[33:33 + t.numel()].view(t.shape)
        guards += [buf[:33], buf[33 + t.numel():]]
    assert torch.equal(c.apply(Y=outs["Y"]), c.apply())
    g = c.grad(out={k: outs[k] for k in ("dX", "dU", "dVt")})
    assert all(torch.equal(g[k], full[k]) for k in full)
    assert all(bool((x == 123).all()) for x in guards)


@pytest.mark.parametrize("b", [20, 150])
def test_non_finite_values_stay_with_their_row_or_adapter(H, b):
    import torch
    c, e = Case(H, 70, 90, 18, b, 4, "each"), Case(H, 70, 90, 18, b, 4, "each")
    rows = np.flatnonzero(c.ids == 1)
    e.d["X"][int(rows[2]), 5] = float("nan")
    Y, Z = c.apply(), e.apply()
    hit = torch.zeros(b, dtype=torch.bool, device="cuda")
    hit[int(rows[2])] = True
    assert not torch.isfinite(Z[hit]).any() and torch.equal(Y[~hit], Z[~hit])
    g, h = c.grad(), e.grad()
    assert torch.equal(g["dX"], h["dX"])                               # does not depend on X
    assert torch.equal(g["dU"][[0, 2, 3]], h["dU"][[0, 2, 3]]) and not torch.isfinite(h["dU"][1]).any()
    only = torch.ones(90, dtype=torch.bool, device="cuda")
    only[5] = False
    assert torch.equal(g["dVt"][[0, 2, 3]], h["dVt"][[0, 2, 3]]) and torch.equal(g["dVt"][1][:, only], h["dVt"][1][:, only])
    assert not torch.isfinite(h["dVt"][1][:, 5]).any()
    # an adapter whose factors are not finite leaves the others' rows alone
    e = Case(H, 70, 90, 18, b, 4, "each")
    e.d["U"][2].fill_(float("inf"))
    e.d["Vt"][2].fill_(float("nan"))
    Z, h = e.apply(), e.grad()
    keep = torch.from_numpy(c.ids != 2).cuda()
    assert torch.equal(Y[keep], Z[keep]) and torch.equal(g["dX"][keep], h["dX"][keep])
    assert torch.equal(g["dU"][[0, 1, 3]], h["dU"][[0, 1, 3]]) and torch.equal(g["dVt"][[0, 1, 3]], h["dVt"][[0, 1, 3]])
    assert not torch.isfinite(Z[~keep]).any()


def test_a_workspace_serves_smaller_batches(H):
    import torch
    top = Case(H, 300, 700, 40, 500, 5, "mixed")
    ws = _nan_ws(H.hss_adapters_workspace_size(top.L, 500))
    gws = _nan_ws(H.hss_adapters_grad_workspace_size(top.L, 500))
    for b in (1, 16, 64, 65, 200, 500):
        X, G, ids = top.d["X"][:b], top.d["G"][:b], top.ids_d[:b].contiguous()
        assert torch.equal(H.hss_adapters_apply(top.L, X, ids, ws=ws), H.hss_adapters_apply(top.L, X, ids))
        a, e = H.hss_adapters_grad(top.L, X, G, ids, ws=gws), H.hss_adapters_grad(top.L, X, G, ids)
        assert all(torch.equal(a[k], e[k]) for k in e)


def test_same_bits_again_and_on_another_stream(H):
    import torch
    c = Case(H, 300, 700, 40, 333, 5, "mixed")
    want = [c.apply(), *c.grad().values()]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = [c.apply(), *c.grad().values()]
    torch.cuda.synchronize()
    assert all(torch.equal(a, w) for a, w in zip(got, want))


@pytest.mark.parametrize("b", [8, 100])
def test_graph_replays_with_new_rows_and_ids(H, b):
    """Forward and backward captured once, replayed with other inputs and other
    adapters for the rows, eager work in between."""
    import torch
    c = Case(H, 160, 224, 24, b, 6, "mixed")
    Y = torch.empty_like(c.d["base"])
    out = {k: torch.empty_like(v) for k, v in c.grad().items()}
    ws, gws = H.adapters_workspace(c.L, b, "cuda"), H.adapters_grad_workspace(c.L, b, "cuda")
    c.apply(Y=Y, ws=ws), c.grad(out=out, ws=gws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.apply(Y=Y, ws=ws)
        c.grad(out=out, ws=gws)
    for rep, kind in enumerate(("one", "mixed", "each", "none")):
        c.d["X"].copy_(to_dev(_rand((b, 224), rep + 50, 1.0), BF))
        c.d["G"].copy_(to_dev(_rand((b, 160), rep + 60, 1.0), BF))
        c.ids_d.copy_(torch.from_numpy(_ids(kind, b, 6, rep).astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        got = [Y.clone()] + [out[k].clone() for k in ("dX", "dU", "dVt")]
        want = [c.apply()] + [c.grad()[k] for k in ("dX", "dU", "dVt")]
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip(got, want)), kind


@pytest.mark.parametrize("b", [12, 80])
def test_gradients_against_differences(H, b):
    """dX, dU and dVt along random directions against the forward's own central
    differences (the forward is linear in each): its outputs' bounds, weighed by
    |G|, over the step, and the gradient's own bound."""
    c = Case(H, 48, 72, 10, b, 3, "mixed", based=False)
    want, tol = c.grad_bounds()
    g = {k: v.double().cpu().numpy() for k, v in c.grad().items()}
    for key, name in (("dX", "X"), ("dU", "U"), ("dVt", "Vt")):
        rng = np.random.default_rng(3)
        D = np.sign(rng.standard_normal(c.f[name].shape)) * 0.5
        total, slack = 0.0, 0.0
        held, kept = c.f[name], c.d[name].clone()
        for s in (1, -1):
            import torch
            moved = torch.from_numpy(held + s * D).to(torch.bfloat16)
            c.d[name].copy_(moved)
            c.f[name] = moved.double().numpy()
            total += s * float(np.sum(c.f["G"] * c.apply().double().cpu().numpy()))
            slack += float(np.sum(np.abs(c.f["G"]) * c.apply_bound()[1]))
            if s == 1:
                step = c.f[name].copy()
        step = (step - c.f[name])
        c.f[name] = held
        c.d[name].copy_(kept)
        assert abs(total - float(np.sum(g[key] * step))) <= slack + float(np.sum(tol[key] * np.abs(step)))


def test_beside_a_compressed_layer(H):
    """A training step of adapters beside a frozen compressed layer: forward,
    backward and AdamW, then the forward again.  Each call against the oracle,
    from what the call before it returned."""
    import torch
    m, n, r, b, count = 200, 160, 12, 70, 3
    sp = H.hss_split(to_dev(syn.random_matrix(m, n, BF, seed=1, kind="t3"), BF), "csr", frac=(5, 100))
    U, V = syn.factors(m, n, 20, BF, 2)
    A = H.HSSMatrix.from_split(sp, U=to_dev(U, BF), Vt=to_dev(np.ascontiguousarray(V.T), BF))
    At = H.hss_transposed_layer(A)
    c = Case(H, m, n, r, b, count, "mixed", seed=5)
    state = H.AdamWState([c.L.U, c.L.Vt], bits=8, master=True)
    before = None
    for t in (1, 2):
        shared = H.hss_apply(A, c.d["X"])
        c.d["base"] = shared
        c.f["base"] = O.widen(to_host(shared), BF)
        Y = c.apply()
        c.check_apply(Y)
        assert before is None or not torch.equal(Y, before)
        before = Y
        dX = H.hss_apply(At, c.d["G"])
        c.d["dbase"], c.f["dbase"] = dX, O.widen(to_host(dX), BF)
        g = c.grad()
        c.check_grad(g)
        master = [w.clone() for w in state.master]
        H.hss_adamw(state, [g["dU"], g["dVt"]], lr=1e-2, step=t)
        assert all(not torch.equal(a, w) for a, w in zip(master, state.master))
        for k, (w, p) in enumerate(zip(state.master, (c.L.U, c.L.Vt))):
            assert torch.equal(w.bfloat16(), p.view(-1))
            c.f[("U", "Vt")[k]] = p.double().cpu().numpy()


def test_a_decode_batch_and_a_prefill_at_full_size(H):
    """4096 x 11008 with 64 requests of their own, and 2048 rows of four: a few
    rows and columns of each against the oracle."""
    for b, count, kind in ((64, 64, "each"), (2048, 4, "runs")):
        c = Case(H, 4096, 11008, 64, b, count, kind)
        Y, g = c.apply(), c.grad()
        rows = np.arange(0, b, max(1, b // 24))
        sub = Case.__new__(Case)
        sub.__dict__.update(c.__dict__, ids=c.ids[rows], b=b)
        sub.f = dict(c.f, **{k: c.f[k][rows] for k in ("X", "G", "base", "dbase")})
        want, tol = sub.apply_bound()
        assert np.all(np.abs(Y.double().cpu().numpy()[rows] - want) <= tol)
        want, tol = sub.grad_bounds()
        assert np.all(np.abs(g["dX"].double().cpu().numpy()[rows] - want["dX"]) <= tol["dX"])
        # dU and dVt of one adapter at a few columns: the others' columns and adapters left out of the oracle
        l, js = int(c.ids[0]), np.arange(3, 4096, 257)
        mine = np.flatnonzero(c.ids == l)
        T, P = c.f["X"][mine] @ c.f["Vt"][l].T, c.f["G"][mine] @ c.f["U"][l]
        aT, aP = np.abs(c.f["X"][mine]) @ np.abs(c.f["Vt"][l]).T, np.abs(c.f["G"][mine]) @ np.abs(c.f["U"][l])
        s = float(c.scale[l])
        for got, want, N, K in ((g["dU"][l, js], s * c.f["G"][mine][:, js].T @ T, abs(s) * np.abs(c.f["G"][mine][:, js]).T @ aT, 11008),
                                (g["dVt"][l][:, js], s * P.T @ c.f["X"][mine][:, js], abs(s) * aP.T @ np.abs(c.f["X"][mine][:, js]), 4096)):
            assert np.all(np.abs(got.double().cpu().numpy() - want) <= 1.01 * (K + 3 * len(mine) + 3) * U24 * N)


@pytest.mark.parametrize("b,m,n,r", [(1, 600, 600, 8), (64, 600, 600, 40), (5, 1100, 1100, 3), (70, 600, 600, 20), (70, 1100, 1300, 65)])
def test_finite_products_past_the_largest_bf16(H, b, m, n, r):
    """T and P of 2^128 - 2^118, a finite fp32 that bf16 rounds to infinity, times 2^-100 of the next
    factor: outputs of 2^28 (1 - 2^-10), not infinities."""
    import torch
    top = [2.0 ** 128 - 2.0 ** 120, 2.0 ** 119, 2.0 ** 118]
    scale = np.array([1.0, -1.0], np.float32)
    ids = np.arange(b) % 2
    tall = lambda shape: np.broadcast_to(np.array(top + [0.0] * (shape[1] - 3)), shape)   # noqa: E731
    first = np.zeros(r)
    first[r - 1] = 1.0
    for grad in (False, True):
        # forward: X tall, Vt ones, U 2^-100; dU of it with G 2^-100.  Backward: G tall, U ones, Vt and X 2^-100
        X = np.full((b, n), 2.0 ** -100) if grad else tall((b, n))
        G = tall((b, m)) if grad else np.full((b, m), 2.0 ** -100)
        U = np.broadcast_to(first * (1.0 if grad else 2.0 ** -100), (2, m, r))
        Vt = np.broadcast_to((first * (2.0 ** -100 if grad else 1.0))[:, None], (2, r, n))
        dev = [torch.from_numpy(np.array(a, order="C")).to("cuda", torch.bfloat16) for a in (U, Vt, X, G)]
        assert all(np.array_equal(t.double().cpu().numpy(), a) for t, a in zip(dev, (U, Vt, X, G)))
        L = H.HSSAdapters(dev[0], dev[1], torch.from_numpy(scale).cuda())
        ids_d = torch.from_numpy(ids.astype(np.int32)).cuda()
        want = O.adapters_grad(U, Vt, scale.astype(np.float64), X, G, ids)
        got = H.hss_adapters_grad(L, dev[2], dev[3], ids_d, dX=grad, dU=not grad, dVt=grad)
        # every sum has terms of one sign: as at the top, with |value| for N
        for key, w, bound in (("dX", want[0], 2.0 ** -8 + (m + 2 * r + 3) * U24 + 2.0 ** -16), ("dU", want[1], (n + 3 * b + 3) * U24),
                              ("dVt", want[2], (m + 3 * b + 3) * U24)):
            if key in got:
                assert np.all(np.abs(got[key].double().cpu().numpy() - w) <= 1.01 * bound * np.abs(w)), key
        if not grad:
            Y = H.hss_adapters_apply(L, dev[2], ids_d).double().cpu().numpy()
            want = O.adapters_apply(U, Vt, scale.astype(np.float64), X, ids)
            assert np.all(np.abs(Y - want) <= 1.01 * (2.0 ** -8 + (n + 2 * r + 3) * U24 + 2.0 ** -16) * np.abs(want))


@pytest.mark.parametrize("m,n,r,b,count,kind", [
    (11003, 520, 9, 64, 64, "each"), (5003, 520, 16, 64, 9, "mixed"), (11003, 517, 32, 64, 12, "mixed"),
    (5003, 520, 32, 64, 64, "each"), (11003, 520, 16, 40, 7, "one"), (16384, 64, 8, 64, 5, "mixed")])
@pytest.mark.parametrize("based", [True, False])
def test_one_launch_of_many_column_blocks(H, m, n, r, b, count, kind, based):
    """Few rows and small factors, more column blocks than compute units (ceil(m / 512) b > 256): a
    block goes through 2 to 8 times 512 columns, with and without base, and in place."""
    import torch
    c = Case(H, m, n, r, b, count, kind, seed=m + r, based=based)
    Y = c.apply()
    c.check_apply(Y)
    if based:
        again = c.d["base"].clone()
        H.hss_adapters_apply(c.L, c.d["X"], c.ids_d, base=again, Y=again)
        assert torch.equal(again, Y)


@pytest.mark.parametrize("m,n,r,b,count,kind", [
    (4099, 200, 40, 64, 64, "each"), (4099, 200, 40, 2048, 3, "mixed"), (11003, 96, 33, 2048, 5, "runs"),
    (4099, 130, 300, 2048, 3, "mixed"), (4610, 130, 5, 2048, 2, "mixed"), (65539, 72, 257, 64, 2, "mixed")])
@pytest.mark.parametrize("based", [True, False])
def test_many_column_blocks_a_tile(H, m, n, r, b, count, kind, based):
    """ceil(m / 512) times the busy tiles >= 512: a block goes through several times 512 columns, the
    last of them ragged, with ranks that are kept in LDS at once and ranks (past 256) that are not."""
    import torch
    c = Case(H, m, n, r, b, count, kind, seed=m + r, based=based)
    Y = c.apply(ws=_nan_ws(H.hss_adapters_workspace_size(c.L, b)))
    c.check_apply(Y)
    if based:
        again = c.d["base"].clone()
        H.hss_adapters_apply(c.L, c.d["X"], c.ids_d, base=again, Y=again)
        assert torch.equal(again, Y)


@pytest.mark.parametrize("m,n,r,count", [(4, 257, 33, 64), (5, 300, 64, 40), (258, 4, 200, 20), (700, 5, 49, 33), (4, 4, 64, 60)])
@pytest.mark.parametrize("b,kind", [(65, "mixed"), (300, "runs"), (515, "one")])
def test_shared_terms_with_rows_of_four_columns(H, m, n, r, count, b, kind):
    """The shortest rows that the blocks of 256 columns take, of which most lanes have none."""
    import torch
    c = Case(H, m, n, r, b, count, kind, seed=r + b, shift=b % 2)
    full = c.grad(ws=_nan_ws(H.hss_adapters_grad_workspace_size(c.L, b)))
    c.check_grad(full)
    for keys in (("dU",), ("dVt",)):
        got = c.grad(**{k: k in keys for k in ("dX", "dU", "dVt")})
        assert all(torch.equal(got[k], full[k]) for k in keys)


@pytest.mark.parametrize("m,n,r,b,count,kind", [(11008, 4096, 64, 2048, 8, "runs"), (11008, 4096, 64, 2048, 8, "one"),
                                                (4096, 4096, 16, 2048, 1, "one")])
def test_same_bits_again_at_full_size(H, m, n, r, b, count, kind):
    """One call after another without a wait, another input's between them, one workspace for all."""
    import torch
    a, o = (Case(H, m, n, r, b, count, kind, seed=s) for s in (1, 20))
    ws, gws = H.adapters_workspace(a.L, b, "cuda"), H.adapters_grad_workspace(a.L, b, "cuda")
    want = [a.apply(), *a.grad().values()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [a.apply(ws=ws), *a.grad(ws=gws).values()]
        o.apply(ws=ws), o.grad(ws=gws)
        assert all(torch.equal(x, w) for x, w in zip(got, want))


@pytest.mark.parametrize("m,n,r,b,count,kind", [
    (4100, 3001, 200, 700, 1, "one"), (4100, 3001, 300, 700, 1, "one"), (4100, 3001, 200, 600, 1, "one"),
    (5003, 4099, 65, 1300, 2, "runs"), (5003, 4099, 130, 1300, 2, "mixed")])
def test_gradients_of_many_rows_an_adapter(H, m, n, r, b, count, kind):
    """On both sides of where their blocks share the terms: 96 blocks of 256 columns up to 640 rows an adapter,
    136 beyond (here 116, 145, 116, 148 and 222)."""
    c = Case(H, m, n, r, b, count, kind, seed=r + b)
    c.check_grad(c.grad(ws=_nan_ws(H.hss_adapters_grad_workspace_size(c.L, b))))
