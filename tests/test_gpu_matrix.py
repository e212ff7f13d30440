"""orthogonalize and muon_step on the GPU against their definitions in 64 bits.

Tolerances (derived, not fitted).  One step X' = P(X X^T) X commutes with the
singular vectors and acts on a singular value as p(s) = a s + b s^3 + c s^5;
in the Frobenius norm such a map is Lipschitz with the largest of |p'(s)|
and |p(s) / s|, 3.9 for the default coefficients and s <= 1.21.  A relative
rounding error eta of the operands of a step moves X' by at most
(|a| + 3 |b| s^2 + 5 |c| s^4) eta |X|_F <= 46 eta |X|_F, and |X_k|_F falls
short of |y|_F by about 3.4 per earlier step, so the last of five iterates is
off by at most about 46 eta (1 + 3.9/3.4 + ...) / 3.4 < 46 * 2.5 eta = 115 eta
of |y|_F.
  full  operands keep 22 bits (two roundings of 2^-23 in a product) and an
        FP32 sum over K values takes 3 K / 16 roundings of 2^-24 in random
        directions: eta = 2^-22 + 2^-24 sqrt(3 K / 16);
  half  S and the polynomial are rounded to 11 bits: at most 2^-12 each,
        2^-12 / sqrt(3) in the root mean square: eta = 2^-12 / sqrt(3).
Smaller side up to 64: FP64 to the end, whose errors (2^-53, growing with the
square of the amplification, at most 3.45^10 = 2.4e5) stay below 1e-9.
Storing y rounds once, by half a step at most: FP32 has 24 significant bits,
so neighbours in [1, 2) are 2^-23 apart and the rounding is at most 2^-24 of
the value; BF16 has 8 bits, neighbours 2^-7 apart, at most 2^-8."""
import ctypes
import math

import numpy as np
import pytest

import layer_streamed_optimizer_amd as lso

from gpu_util import log, torch

pytestmark = pytest.mark.gpu

COEF = (3.4445, -4.7750, 2.0315)
CANARY = 0xA5


def ortho64(x, steps=5, eps=1e-7, coef=COEF):
    """The definition, in 64 bits on the CPU."""
    x = np.asarray(x, np.float64)
    if x.shape[0] > x.shape[1]:
        return ortho64(x.T, steps, eps, coef).T
    coef = np.broadcast_to(np.asarray(coef, np.float64), (steps, 3))
    x = x / (np.sqrt((x * x).sum()) + eps)
    for a, b, c in coef:
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    return x


def matrix(rows, cols, seed, kind="noise"):
    rng = np.random.default_rng(seed)
    g = rng.standard_normal((rows, cols)) * 1e-3
    if kind == "spiked":   # a few directions above the noise, as momentum has
        for r in range(4):
            g += np.outer(rng.standard_normal(rows), rng.standard_normal(cols)) * 4e-3 / 2**r
    return g.astype(np.float32)


def small(rows, cols):
    return min(rows, cols) <= 32


def tolerance(rows, cols, full, out_bf16):
    k = max(rows, cols) + 128
    eta = 2.0**-22 + 2.0**-24 * math.sqrt(3 * k / 16) if full else 2.0**-12 / math.sqrt(3)
    return (2e-9 if small(rows, cols) else 115 * eta) + (2.0**-8 if out_bf16 else 2.0**-24)


def check(got, want, rows, cols, full, out_bf16, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    tol = tolerance(rows, cols, full, out_bf16)
    norm = np.linalg.norm(want)
    err = np.linalg.norm(got - want) / norm if norm else np.linalg.norm(got)
    assert err <= tol, f"{what}: relative error {err:.3g} > {tol:.3g}"
    # no single element may hide in the norm: errors are spread over the
    # matrix, so one is at most a few times its share of the whole
    worst = np.max(np.abs(got - want)) if got.size else 0.0
    share = tol * norm / math.sqrt(got.size) if got.size else 0.0
    step = (2.0**-8 if out_bf16 else 2.0**-24) * (np.max(np.abs(want)) if got.size else 0.0)
    assert worst <= 12 * share + step, f"{what}: an element is off by {worst:.3g}, share {share:.3g}"


class Mats:
    """Inputs and results of a call, each in a buffer of its own with canary
    bytes around it and between its rows."""

    def __init__(self, shapes, x_dtype="f32", y_dtype="f32", pad_x=0, pad_y=0, kind="noise", seed=0, shift=0):
        T = torch()
        self.shapes, self.x, self.y, self.src = shapes, [], [], []
        td = {"f32": T.float32, "bf16": T.bfloat16}
        for i, (r, c) in enumerate(shapes):
            bufs = []
            for dt, pad in ((x_dtype, pad_x), (y_dtype, pad_y)):
                es = 4 if dt == "f32" else 2
                raw = T.full(((r * (c + pad) + 64 + shift) * es,), CANARY, dtype=T.uint8, device="cuda")
                bufs.append(raw.view(td[dt])[32 + shift:32 + shift + r * (c + pad)].view(r, c + pad)[:, :c])
                bufs.append(raw)
            x, xr, y, yr = bufs
            x.copy_(T.from_numpy(matrix(r, c, seed + i, kind)))
            self.x.append((x, xr))
            self.y.append((y, yr))
            self.src.append(x.float().cpu().numpy())
        self.ids = (x_dtype, y_dtype, pad_x, pad_y)
        self.table = lso.MatrixTable.from_rows(
            dict(x=x, y=y, rows=r, cols=c, ld_x=c + pad_x, ld_y=c + pad_y, x_dtype=1 if x_dtype == "f32" else 2,
                 y_dtype=1 if y_dtype == "f32" else 2) for (r, c), (x, _), (y, _) in zip(shapes, self.x, self.y))

    def results(self):
        return [y.float().cpu().numpy() for y, _ in self.y]

    def check_canaries(self):
        for (r, c), (y, raw) in zip(self.shapes, self.y):
            host = raw.cpu().clone()
            dst = host.view(y.dtype)
            off = y.storage_offset()
            dst[off:off + r * y.stride(0)].view(r, y.stride(0))[:, :c].zero_()
            want = torch().full_like(host, CANARY)
            want.view(y.dtype)[off:off + r * y.stride(0)].view(r, y.stride(0))[:, :c].zero_()
            assert torch().equal(host, want), f"written outside {r} x {c}"


def workspace(nbytes, slack=512):
    """Device workspace with a canary band behind it, filled with NaN-like bytes."""
    ws = torch().full((nbytes + slack,), 0xFF, dtype=torch().uint8, device="cuda")
    ws[nbytes:] = CANARY
    return ws


def run_ortho(m, **kw):
    need = lso.orthogonalize_workspace_bytes(m.table, kw.get("precision", 0))
    ws = workspace(need)
    lso.orthogonalize(m.table, ws, need, **kw)
    torch().cuda.synchronize()
    assert bool((ws[need:] == CANARY).all()), "written behind the workspace"
    m.check_canaries()
    return m.results()


SHAPES = [(1, 1), (1, 7), (7, 1), (8, 8), (9, 300), (300, 9), (16, 17), (31, 1000), (32, 32), (2049, 32), (33, 33), (64, 65),
          (127, 129), (128, 128), (129, 40), (200, 500), (500, 200), (256, 2048)]


@pytest.mark.parametrize("precision", [lso.LSO_NS_FULL, lso.LSO_NS_HALF])
@pytest.mark.parametrize("x_dtype,y_dtype", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_orthogonalize_shapes_in_one_call(precision, x_dtype, y_dtype):
    log(f"orthogonalize {x_dtype} -> {y_dtype}, precision {precision}, {len(SHAPES)} shapes")
    m = Mats(SHAPES, x_dtype, y_dtype, pad_x=5, pad_y=3)
    for (r, c), src, got in zip(SHAPES, m.src, run_ortho(m, precision=precision)):
        check(got, ortho64(src), r, c, precision == lso.LSO_NS_FULL, y_dtype == "bf16", f"{r}x{c}")


@pytest.mark.parametrize("precision", [lso.LSO_NS_FULL, lso.LSO_NS_HALF])
@pytest.mark.parametrize("kind", ["noise", "spiked"])
def test_orthogonalize_sides_of_33_to_64_in_fp64(precision, kind):
    """Smaller sides of 33 to 64 go the way of 32 and less, FP64 to the end
    whatever the precision, alone and where they are long enough next to
    larger matrices; a few of them go with the larger ones."""
    few = [(33, 33), (33, 257), (64, 64), (64, 2048), (1000, 64), (63, 513), (48, 16384), (2049, 40), (40, 16385), (5, 9)]
    for shapes, fp64 in ((few, True), (few + [(65, 100)], False), (few + [(30000, 40), (65, 100)], True)):
        m = Mats(shapes, kind=kind, seed=17, pad_x=3, pad_y=1)
        log(f"orthogonalize sides of 33 to 64, precision {precision}, {kind}, {len(shapes)} matrices")
        for (r, c), src, got in zip(shapes, m.src, run_ortho(m, precision=precision)):
            want = ortho64(src)
            err = np.linalg.norm(got - want) / np.linalg.norm(want)
            # twice the side of 32: twice the terms of a sum, under 4e-9 by the same count
            allow = 4e-9 + 2.0**-24 if fp64 and min(r, c) <= 64 else tolerance(r, c, precision == lso.LSO_NS_FULL, False)
            assert err <= allow, (r, c, err, allow)


@pytest.mark.parametrize("rows,cols", [(8, 2048), (5632, 8), (40, 4099), (700, 300), (384, 1024)])
@pytest.mark.parametrize("kind", ["noise", "spiked"])
def test_orthogonalize_alone_auto_precision(rows, cols, kind):
    for xd, yd in (("f32", "f32"), ("bf16", "bf16")):
        log(f"orthogonalize alone {rows}x{cols} {kind} {xd}")
        m = Mats([(rows, cols)], xd, yd, kind=kind, seed=7, shift=1)
        got = run_ortho(m)[0]
        check(got, ortho64(m.src[0]), rows, cols, yd == "f32", yd == "bf16", f"{rows}x{cols} {kind} {xd}")


def test_orthogonalize_steps_eps_and_coefficients():
    shapes = [(20, 50), (100, 150)]
    triples = [(1.5, -0.5, 0.0), (3.4445, -4.7750, 2.0315), (1.875, -1.25, 0.375)]
    for kw, ref in ((dict(steps=1), {}), (dict(steps=3, eps=0.5), dict(eps=0.5)), (dict(steps=3, coefficients=triples), dict(coef=triples)),
                    (dict(steps=16, coefficients=(1.5, -0.5, 0.0)), dict(coef=(1.5, -0.5, 0.0)))):
        log(f"orthogonalize {kw}")
        m = Mats(shapes, seed=11)
        for (r, c), src, got in zip(shapes, m.src, run_ortho(m, **kw)):
            # these maps have smaller Lipschitz constants than the default; up to 16 steps instead of 5
            want = ortho64(src, kw["steps"], ref.get("eps", 1e-7), ref.get("coef", COEF))
            err = np.linalg.norm(got - want) / np.linalg.norm(want)
            assert err <= 4 * tolerance(r, c, True, False), (kw, r, c, err)


def ortho64_gpu(x, steps=5, coef=COEF):
    x = x.double()
    if x.shape[0] > x.shape[1]:
        return ortho64_gpu(x.T.contiguous(), steps, coef).T
    x = x / (x.norm() + 1e-7)
    for a, b, c in np.broadcast_to(np.asarray(coef, np.float64), (steps, 3)):
        s = x @ x.T.contiguous()
        x = float(a) * x + (float(b) * s + float(c) * (s @ s)) @ x
    return x


@pytest.mark.parametrize("shapes", [
    [(300, 9001), (70, 4000)],          # long: steps in pairs, tiles of 64
    [(2050, 2311)],                     # nearly square: single steps, tiles of 64
    [(777, 9000), (9001, 1030)],        # steps in pairs, tiles of 64
    [(4099, 4501)],                     # tiles of 128, single steps
    [(12001, 3001)],                    # tiles of 128, steps in pairs
    [(5050, 5070)],                     # tiles of 256, single steps
    [(16001, 4090), (257, 300)],        # tiles of 256, steps in pairs
])
@pytest.mark.parametrize("precision", [lso.LSO_NS_FULL, lso.LSO_NS_HALF])
def test_orthogonalize_large(shapes, precision):
    T = torch()
    T.manual_seed(5)
    xs = [T.randn(r, c, device="cuda") + 3.0 * T.outer(T.randn(r, device="cuda"), T.randn(c, device="cuda")) for r, c in shapes]
    ys = [T.full_like(x, 7.0) for x in xs]
    table = lso.MatrixTable.from_rows(dict(x=x, y=y, rows=x.shape[0], cols=x.shape[1]) for x, y in zip(xs, ys))
    need = lso.orthogonalize_workspace_bytes(table, precision)
    ws = workspace(need)
    for steps in (5, 1, 4):
        log(f"orthogonalize large {shapes} precision {precision} steps {steps}")
        lso.orthogonalize(table, ws, need, steps=steps, precision=precision)
        T.cuda.synchronize()
        assert bool((ws[need:] == CANARY).all())
        for x, y in zip(xs, ys):
            want = ortho64_gpu(x, steps)
            err = float((y.double() - want).norm() / want.norm())
            assert err <= tolerance(*x.shape, precision == lso.LSO_NS_FULL, False), (x.shape, steps, err)
            share = tolerance(*x.shape, precision == lso.LSO_NS_FULL, False) * float(want.norm()) / math.sqrt(want.numel())
            assert float((y.double() - want).abs().max()) <= 12 * share


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6])
@pytest.mark.parametrize("precision", [lso.LSO_NS_FULL, lso.LSO_NS_HALF])
def test_orthogonalize_steps_in_pairs(steps, precision):
    """Every way that a number of steps is taken in pairs and singly, with
    coefficients that allow pairs everywhere, nowhere and in places (a pair is
    taken where the product of its two polynomials stays in FP16's range)."""
    shapes = [(50, 3000), (3000, 90)]
    mild, steep = (1.5, -0.5, 0.0), (8.0, -20.0, 13.0)   # 1.5 x 8 < 15.9 < 8 x 8
    for coef in ([mild] * steps, [steep] + [mild] * (steps - 1), [mild if k % 3 else steep for k in range(steps)]):
        m = Mats(shapes, seed=60 + steps)
        log(f"orthogonalize in pairs: {steps} steps, precision {precision}, {coef}")
        for (r, c), src, got in zip(shapes, m.src, run_ortho(m, steps=steps, coefficients=coef, precision=precision)):
            want = ortho64(src, steps, coef=coef)
            # steep steps: Lipschitz constant 8 where the default's is 3.9, and (8 + 3 20 s^2 + 5 13 s^4) / 46 < 3 times
            # its rounding, for at most two of six steps
            allow = 3 * (8 / 3.9)**2 * tolerance(r, c, precision == lso.LSO_NS_FULL, False)
            err = np.linalg.norm(got - want) / np.linalg.norm(want)
            assert err <= allow, (r, c, coef, err, allow)


def test_orthogonalize_extreme_values():
    """Zero matrices, one element, tiny and huge scales (|u|_F is summed in
    FP64), and a NaN or an infinity that stays in its own matrix."""
    shapes = [(40, 50), (40, 50), (40, 50), (40, 50), (40, 50), (40, 50), (10, 50), (10, 50), (10, 50), (10, 50)]
    m = Mats(shapes, seed=3)
    edits = {0: 0.0, 1: 1e-30, 2: 1e30, 6: 0.0, 7: 1e30}
    for i, f in edits.items():
        m.x[i][0].mul_(f)
    m.x[3][0][3, 4] = float("nan")
    m.x[4][0][39, 49] = float("inf")
    m.x[8][0][3, 4] = float("nan")
    src = [x.cpu().numpy() for x, _ in m.x]
    log("orthogonalize extreme values")
    got = run_ortho(m)
    for i in (0, 6):
        assert not got[i].any()
    for i in (1, 2, 5, 7, 9):
        check(got[i], ortho64(src[i]), *shapes[i], True, False, f"matrix {i}")
    for i in (3, 4, 8):
        assert np.isnan(got[i]).any()


def test_orthogonalize_in_place_and_repeatable():
    shapes = [(12, 700), (700, 12), (150, 260), (260, 150)]
    for dt in ("f32", "bf16"):
        a, b = Mats(shapes, dt, dt, seed=5), Mats(shapes, dt, dt, seed=5)
        want = run_ortho(a)
        for i in range(len(shapes)):
            b.table.arr["y"][i] = b.table.arr["x"][i]
            b.table.arr["ld_y"][i] = b.table.arr["ld_x"][i]
        need = lso.orthogonalize_workspace_bytes(b.table)
        ws = workspace(need)
        log(f"orthogonalize in place {dt}")
        lso.orthogonalize(b.table, ws, need)
        torch().cuda.synchronize()
        for (x, _), w in zip(b.x, want):
            assert np.array_equal(x.float().cpu().numpy(), w)   # the same bits as out of place, and again


def test_orthogonalize_on_another_stream_and_captured():
    T = torch()
    shapes = [(8, 400), (130, 250)]
    m = Mats(shapes, seed=9)
    want = run_ortho(m)
    need = lso.orthogonalize_workspace_bytes(m.table)
    s = T.cuda.Stream()
    for (y, _) in m.y:
        y.zero_()
    ws = [workspace(need), workspace(need)]
    T.cuda.synchronize()
    log("orthogonalize on a stream")
    with T.cuda.stream(s):
        lso.orthogonalize(m.table, ws[0], need)
    s.synchronize()
    for g, w in zip(m.results(), want):
        assert np.array_equal(g, w)
    log("orthogonalize captured")
    g = T.cuda.CUDAGraph()
    with T.cuda.graph(g):
        lso.orthogonalize(m.table, ws[1], need)
    for k in range(3):
        # new inputs of the same buffers, an eager call between the replays
        for i, (x, _) in enumerate(m.x):
            x.copy_(T.from_numpy(matrix(*shapes[i], 100 + 10 * k + i)))
        for (y, _) in m.y:
            y.zero_()
        g.replay()
        T.cuda.synchronize()
        got = m.results()
        for (y, _) in m.y:
            y.zero_()
        lso.orthogonalize(m.table, ws[0], need)
        T.cuda.synchronize()
        for a, b in zip(got, m.results()):
            assert np.array_equal(a, b) and a.any()


# ------------------------------------------------------------------- the update

def bf16(a):
    """FP32 -> BF16 bits, to nearest even."""
    u = np.ascontiguousarray(a, np.float32).view(np.uint32)
    return ((u.astype(np.uint64) + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


class Block:
    """Matrices back to back in flat arrays (as in a layer block), with one
    canary element behind each array."""

    def __init__(self, shapes, grad="bf16", weight=True, seed=0, shift=0, **hyper):
        T = torch()
        self.shapes, self.weight, self.hyper = shapes, weight, hyper
        n = sum(r * c for r, c in shapes)
        rng = np.random.default_rng(seed)
        g = np.concatenate([matrix(r, c, seed + 1 + i, "spiked").ravel() for i, (r, c) in enumerate(shapes)])
        self.host = dict(master=(rng.standard_normal(n) * 0.02).astype(np.float32),
                         m=(0.5 * g + 1e-3 * rng.standard_normal(n)).astype(np.float32), grad=g)
        self.n, self.shift = n, shift

        def dev(a, dt):
            t = T.zeros(n + shift + 1, dtype=dt, device="cuda")
            t[shift:shift + n] = T.from_numpy(a)
            t[shift + n:] = 77.0
            return t
        self.master, self.m = dev(self.host["master"], T.float32), dev(self.host["m"], T.float32)
        self.grad = dev(g, T.float32 if grad == "f32" else T.bfloat16)
        self.w = dev(np.zeros(n, np.float32), T.bfloat16) if weight else None
        self.host["grad"] = self.grad[shift:shift + n].float().cpu().numpy()
        rows, at = [], shift
        for i, (r, c) in enumerate(shapes):
            rows.append(dict(rows=r, cols=c, master=self.master.data_ptr() + 4 * at, m=self.m.data_ptr() + 4 * at,
                             grad=self.grad.data_ptr() + (4 if grad == "f32" else 2) * at, grad_dtype=1 if grad == "f32" else 2,
                             weight=self.w.data_ptr() + 2 * at if weight else None, **hyper))
            at += r * c
        self.table = lso.MuonTable.from_rows(rows)

    def step64(self, full=True):
        """One step of the definition on the host state, in 64 bits, with the
        FP32 constants and the FP32 momentum that the next step starts from."""
        h = dict(lr=1e-3, beta=0.95, weight_decay=0.0, scale=1.0, nesterov=True, **{})
        h.update(self.hyper)
        beta, c1 = np.float64(np.float32(h["beta"])), np.float64(np.float32(1.0 - h["beta"]))
        keep, step = np.float64(np.float32(1.0 - h["lr"] * h["weight_decay"])), np.float64(np.float32(-h["lr"] * h["scale"]))
        g = self.host["grad"].astype(np.float64)
        m = beta * self.host["m"] + c1 * g
        u = beta * m + c1 * g if h["nesterov"] else m
        o, at = np.empty(self.n), 0
        tol = np.empty(self.n)
        for r, c in self.shapes:
            y = ortho64(u[at:at + r * c].reshape(r, c))
            o[at:at + r * c] = y.ravel()
            # u is off by up to three FP32 roundings, which count like one more operand rounding
            t = tolerance(r, c, full, False) + 115 * 2.0**-22
            tol[at:at + r * c] = 12 * t * np.linalg.norm(y) / math.sqrt(r * c) + 2.0**-23 * np.max(np.abs(y))
            at += r * c
        master = keep * self.host["master"] + step * o
        # |m'| : two products and one sum, each rounded; master likewise, plus the step's own error
        m_tol = 2.0**-23 * (np.abs(beta * self.host["m"]) + np.abs(c1 * g)) + 1e-45
        master_tol = 2.0**-23 * (np.abs(keep * self.host["master"]) + np.abs(step * o)) + abs(step) * tol
        return m, m_tol, master, master_tol

    def check(self, full=True, what=""):
        T, s = torch(), slice(self.shift, self.shift + self.n)
        m, m_tol, master, master_tol = self.step64(full)
        got_m, got = self.m[s].cpu().numpy(), self.master[s].cpu().numpy()
        assert np.all(np.abs(got_m - m) <= m_tol), f"{what}: m off by {np.max(np.abs(got_m - m) / m_tol):.3g} of its bound"
        assert np.all(np.abs(got - master) <= master_tol), \
            f"{what}: master off by {np.max(np.abs(got - master) / master_tol):.3g} of its bound"
        if self.w is not None:
            assert np.array_equal(self.w[s].view(T.int16).cpu().numpy().view(np.uint16), bf16(got)), what
        for t in (self.master, self.m, self.grad) + ((self.w,) if self.weight else ()):
            assert float(t[self.shift + self.n]) == 77.0, f"{what}: written behind an array"
            assert not t[:self.shift].any(), f"{what}: written before an array"
        self.host["m"], self.host["master"] = got_m, got


def run_muon(b, **kw):
    need = lso.muon_workspace_bytes(b.table, kw.get("precision", 0))
    ws = workspace(need)
    lso.muon_step(b.table, ws, need, **kw)
    torch().cuda.synchronize()
    assert bool((ws[need:] == CANARY).all())


MUON_SHAPES = [(1, 1), (3, 2), (8, 300), (301, 8), (33, 40), (130, 70), (64, 257), (256, 512)]


@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("shift", [0, 1])
def test_muon_steps(grad, weight, shift):
    b = Block(MUON_SHAPES, grad, weight, seed=20, shift=shift, lr=0.02, beta=0.9, weight_decay=0.1, scale=1.5)
    for k in range(3):
        log(f"muon step {k} grad {grad} weight {weight} shift {shift}")
        run_muon(b)
        b.check(what=f"step {k}")


def test_muon_without_nesterov_beta_zero_and_half_precision():
    for hyper, kw in ((dict(nesterov=False, lr=0.1), {}), (dict(beta=0.0, lr=1.0, scale=0.2), {}), (dict(lr=0.0), {}),
                      (dict(lr=-0.5, beta=0.5), dict(precision=lso.LSO_NS_HALF))):
        log(f"muon {hyper} {kw}")
        b = Block([(5, 9), (100, 140)], "f32", True, seed=31, **hyper)
        run_muon(b, **kw)
        b.check(full=not kw, what=str(hyper))


def test_muon_shared_gradient_and_hyper_parameters_per_matrix():
    b = Block([(40, 60), (40, 60)], "f32", False, seed=40, lr=0.1)
    b.table.arr["off_grad"][1] = b.table.arr["off_grad"][0]
    b.table.arr["lr"][1] = 0.0
    before = b.master.clone()
    log("muon shared gradient")
    run_muon(b)
    half = 40 * 60
    assert not torch().equal(b.master[:half], before[:half])
    assert torch().equal(b.master[half:], before[half:])           # lr 0: the master keeps its bits
    b.host["grad"][half:] = b.host["grad"][:half]
    m, m_tol, _, _ = b.step64()
    assert np.all(np.abs(b.m[:2 * half].cpu().numpy() - m) <= m_tol)


def test_muon_then_adam_over_one_block():
    """A layer as it is trained with both: the matrices by orthogonalised
    momentum, the norm vector behind them by Adam, into one BF16 weight
    array; the whole step captured and replayed against eager steps."""
    T = torch()
    n_norm = 96

    def make():
        b = Block([(96, 96), (96, 160), (20, 96)], "bf16", True, seed=50, lr=0.02)
        vec = {k: T.full((n_norm,), 0.5 if k == "master" else 0.0, dtype=T.float32, device="cuda") for k in ("master", "m", "v")}
        vec["grad"] = T.full((n_norm,), 1e-3, dtype=T.bfloat16, device="cuda")
        vec["weight"] = T.zeros(n_norm, dtype=T.bfloat16, device="cuda")
        adam = lso.BlockTable.from_rows([dict(n=n_norm, t=3, **vec)])
        need = lso.muon_workspace_bytes(b.table)
        return b, vec, adam, workspace(need), need

    def step(x):
        b, _, adam, ws, need = x
        lso.muon_step(b.table, ws, need)
        lso.adam_step_noalloc(adam)
    eager, graphed = make(), make()
    log("muon and adam eager")
    step(eager)
    T.cuda.synchronize()
    eager[0].check(what="eager")
    log("muon and adam captured")
    g = T.cuda.CUDAGraph()
    with T.cuda.graph(g):
        step(graphed)
    for k in range(3):
        g.replay()
        T.cuda.synchronize()
        if k > 0:
            step(eager)
            T.cuda.synchronize()
        for a, b in ((eager[0].master, graphed[0].master), (eager[0].m, graphed[0].m), (eager[0].w, graphed[0].w),
                     (eager[1]["master"], graphed[1]["master"]), (eager[1]["weight"], graphed[1]["weight"])):
            assert T.equal(a, b), f"replay {k}"


def test_many_matrices_in_one_call():
    """More matrices than one launch carries table entries for, of every path."""
    shapes = [(4, 40 + i) for i in range(90)] + [(50, 12), (12, 50), (20, 30), (60, 70)] * 10
    b = Block(shapes, "f32", False, seed=60, lr=0.3)
    log("muon many matrices")
    run_muon(b)
    b.check(what="many")


def test_matrices_of_many_different_sizes():
    """More different sizes than a launch's runs of alike matrices hold, of the
    small and of the general path: workgroups then search the table."""
    shapes = [(3, 270 * i + 5) for i in range(1, 13)] + [(40 + 30 * i, 50 + 70 * i) for i in range(12)]
    for precision in (lso.LSO_NS_FULL, lso.LSO_NS_HALF):
        m = Mats(shapes, seed=80)
        log(f"orthogonalize {len(shapes)} different sizes, precision {precision}")
        for (r, c), src, got in zip(shapes, m.src, run_ortho(m, precision=precision)):
            check(got, ortho64(src), r, c, precision == lso.LSO_NS_FULL, False, f"{r}x{c}")


def test_a_large_table_in_a_graph():
    """As many adapters as a model has, captured: the table travels in the
    arguments of a launch that the graph keeps."""
    T = torch()
    shapes = [(8, 64 + 8 * (i % 5)) for i in range(330)] + [(60, 8)] * 20
    eager, graphed = Block(shapes, "f32", False, seed=90, lr=0.1), Block(shapes, "f32", False, seed=90, lr=0.1)
    need = lso.muon_workspace_bytes(eager.table)
    ws = [workspace(need), workspace(need)]
    log("many adapters eager")
    lso.muon_step(eager.table, ws[0], need)
    T.cuda.synchronize()
    eager.check(what="eager")
    log("many adapters captured")
    g = T.cuda.CUDAGraph()
    with T.cuda.graph(g):
        lso.muon_step(graphed.table, ws[1], need)
    graphed.table.arr["rows"] = 0          # the host table is not read again
    for k in range(3):
        g.replay()
        T.cuda.synchronize()
        if k > 0:
            lso.muon_step(eager.table, ws[0], need)
            T.cuda.synchronize()
        assert T.equal(eager.master, graphed.master) and T.equal(eager.m, graphed.m), f"replay {k}"


def test_two_calls_at_once_on_two_streams():
    """Two calls with workspaces of their own on two streams at once give what
    they give one after the other."""
    T = torch()
    shapes = [[(300, 2000), (8, 900)], [(500, 700), (16, 5000)]]
    want = [run_ortho(Mats(s, seed=95 + i)) for i, s in enumerate(shapes)]
    mats = [Mats(s, seed=95 + i) for i, s in enumerate(shapes)]
    need = [lso.orthogonalize_workspace_bytes(m.table) for m in mats]
    ws = [workspace(n) for n in need]
    streams = [T.cuda.Stream(), T.cuda.Stream()]
    T.cuda.synchronize()
    log("two calls at once")
    for _ in range(3):
        for m, n, w, s in zip(mats, need, ws, streams):
            lso.orthogonalize(m.table, w, n, stream=s)
    T.cuda.synchronize()
    for m, w in zip(mats, want):
        for a, b in zip(m.results(), w):
            assert np.array_equal(a, b)


def test_errors_leave_the_thread_usable():
    lib = lso._native.lib()
    assert lib.lso_muon_step(None, 1, None, None, 0, None) == 1
    b = Block([(10, 20)], "f32", False, seed=70)
    log("muon after an error")
    run_muon(b)
    b.check()
    assert lib.lso_muon_step(ctypes.c_void_p(b.table.ptr), 1, None, None, 0, None) == 1


def test_auto_precision_is_full_for_bf16_results():
    """A BF16 matrix orthogonalised without naming a precision: the bits of
    full precision, and next to nothing but the result's own rounding off the
    definition.  A value within the error e of full precision (its norm-wise
    bound, three times over for a single element) of a midpoint of two BF16
    numbers may round to the other one, a step of 2^-7 of the value at most."""
    shapes = [(256, 500), (900, 200)]
    auto, full = Mats(shapes, "bf16", "bf16", seed=21), Mats(shapes, "bf16", "bf16", seed=21)
    log("orthogonalize BF16 with AUTO and FULL")
    a, f = run_ortho(auto), run_ortho(full, precision=lso.LSO_NS_FULL)
    for (r, c), src, x, y in zip(shapes, auto.src, a, f):
        assert np.array_equal(x, y)
        want = ortho64(src)
        rounded = (bf16(want.astype(np.float32)).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        share = 3 * tolerance(r, c, True, False) * np.linalg.norm(want) / math.sqrt(want.size)
        off = np.abs(x - rounded)
        assert np.all(off <= 2.0**-7 * np.abs(want) + share)


def test_tables_take_type_and_stride_from_tensors():
    """BF16 tensors and column slices given without codes and strides."""
    T = torch()
    log("tables from tensors")
    src = T.from_numpy(matrix(70, 90, 5)).cuda()
    wide = T.full((70, 101), 9.0, device="cuda").bfloat16()
    wide[:, :90] = src
    out = T.full((70, 95), 7.0, device="cuda").bfloat16()
    table = lso.MatrixTable.from_rows([dict(x=wide[:, :90], y=out[:, :90], rows=70, cols=90)])
    assert table.arr[["ld_x", "ld_y", "x_dtype", "y_dtype"]].tolist() == [(101, 95, 2, 2)]
    need = lso.orthogonalize_workspace_bytes(table)
    lso.orthogonalize(table, workspace(need), need)
    T.cuda.synchronize()
    check(out[:, :90].float().cpu().numpy(), ortho64(wide[:, :90].float().cpu().numpy()), 70, 90, True, True, "slices")
    assert bool((out[:, 90:] == 7.0).all())
    b = Block([(70, 90)], "f32", True, seed=6)
    b.table = lso.MuonTable.from_rows([dict(rows=70, cols=90, master=b.master[:-1].view(70, 90), m=b.m[:-1], grad=b.grad[:-1].view(70, 90),
                                            weight=b.w[:-1])])
    assert b.table.arr["grad_dtype"].tolist() == [1]
    log("update from tensors")
    run_muon(b)
    b.check(what="from tensors")


@pytest.mark.parametrize("precision", [lso.LSO_NS_FULL, lso.LSO_NS_HALF])
def test_orthogonalize_with_coefficients_that_shrink(precision):
    """Steps that make X small, alone and before and between others: X keeps
    its bits (its operands are scaled), so errors stay those of any step.  A
    linear step is off by its operands' rounding alone, less than the default
    ones that the tolerance is made for."""
    shapes = [(40, 60), (100, 130), (130, 100), (90, 3000), (1500, 80)]     # the small path, single steps, pairs
    default, tiny, mild = COEF, (0.02, 0.0, 0.0), (0.3, -0.1, 0.0)
    for coef in ([tiny] * 5, [tiny, default, default, default], [default, default, tiny, tiny, default], [mild] * 16, [(1e-30, 0.0, 0.0)],
                 [tiny, (1.5, -0.5, 0.0)] * 3, [(0.0, 0.0, 0.0)] * 2):
        m = Mats(shapes, seed=33)
        log(f"orthogonalize with coefficients that shrink, precision {precision}, {coef}")
        for (r, c), src, got in zip(shapes, m.src, run_ortho(m, steps=len(coef), coefficients=coef, precision=precision)):
            want = ortho64(src, len(coef), coef=coef)
            norm = np.linalg.norm(want)
            assert np.linalg.norm(got - want) <= tolerance(r, c, precision == lso.LSO_NS_FULL, False) * norm, (r, c, coef)
