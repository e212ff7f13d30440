"""The general path of orthogonalize and muon_step where other tests reach the
small one only: unusual values, tiles of 128 and 256 with steps in pairs,
tables of more entries than one launch writes.  Every test first says which
path its calls take, so that another choice of paths cannot empty it.
Tolerances as in test_gpu_matrix.py."""
import math

import numpy as np
import pytest

import layer_streamed_optimizer_amd as lso

from gpu_util import log, torch
from test_gpu_matrix import Block, CANARY, Mats, ortho64, ortho64_gpu, run_muon, run_ortho, tolerance, workspace

pytestmark = pytest.mark.gpu

FULL, HALF = lso.LSO_NS_FULL, lso.LSO_NS_HALF


def planned(shapes, precision):
    torch()      # its HIP runtime is the one to load first
    table = lso.MatrixTable.from_rows(dict(x=1 << 40, y=1 << 40, rows=r, cols=c) for r, c in shapes)
    return lso.orthogonalize_workspace_bytes(table, precision)


def general(shape):
    """Whether a matrix alone takes the general path, the only one whose
    workspace depends on the precision."""
    return planned([shape], FULL) != planned([shape], HALF)


def tile_edge(shapes, precision):
    """The edge of a call's tiles: sides rounded up to it change nothing."""
    def up(edge):
        return [tuple(-(-side // edge) * edge for side in s) for s in shapes]
    assert len({tuple(up(edge)) for edge in (64, 128, 256)}) == 3, "sides that tell the edges apart"
    return max(edge for edge in (64, 128, 256) if planned(up(edge), precision) == planned(shapes, precision))


# --------------------------------------------------------------- unusual values

def unusual(m, shapes):
    """Edits of ten matrices; what each becomes: "zero", "nan" or "value"."""
    for i, f in {0: 0.0, 1: 1e-30, 2: 1e30, 8: 1e-7, 9: 1e-38}.items():    # 9: FP32 subnormals among them
        m.x[i][0].mul_(f)
    r, c = shapes[3]
    m.x[3][0][r // 2, c // 3] = float("nan")
    r, c = shapes[4]
    m.x[4][0][r - 1, c - 1] = float("inf")
    m.x[6][0][0, 0] = float("-inf")
    m.x[7][0].zero_()
    m.x[7][0][3, 5] = 1e-20
    return ["zero", "value", "value", "nan", "nan", "value", "nan", "value", "value", "value"]


@pytest.mark.parametrize("precision", [FULL, HALF])
@pytest.mark.parametrize("sizes", [[(100, 130), (130, 100)], [(90, 3000), (3000, 90)], [(65, 65), (128, 192)]])
def test_unusual_values(precision, sizes):
    """Zeros, subnormals, 1e-30 and 1e30, a single element, and a NaN or an
    infinity that fills its own matrix and no other; with steps taken singly
    and (90 x 3000) in pairs."""
    shapes = sizes * 5
    assert all(general(s) for s in sizes)
    for kw in ({}, dict(eps=0.5), dict(eps=0.0), dict(steps=1)):
        m = Mats(shapes, seed=3)
        kinds = unusual(m, shapes)
        src = [x.cpu().numpy() for x, _ in m.x]
        log(f"unusual values {sizes} precision {precision} {kw}")
        got = run_ortho(m, precision=precision, **kw)
        for i, kind in enumerate(kinds):
            what = f"matrix {i} of {shapes[i]}, {kw}"
            if kind == "nan" or (kind == "zero" and kw.get("eps") == 0.0):
                assert np.isnan(got[i]).all(), what
            elif kind == "zero":
                assert not got[i].any(), what
            else:
                want = ortho64(src[i], kw.get("steps", 5), kw.get("eps", 1e-7))
                err, norm = np.linalg.norm(got[i] - want), np.linalg.norm(want)
                assert norm > 0 and err <= tolerance(*shapes[i], precision == FULL, False) * norm, (what, err / norm)


@pytest.mark.parametrize("shape,edge", [((2100, 5100), 128), ((5100, 2100), 128), ((4100, 16100), 256)])
@pytest.mark.parametrize("precision", [FULL, HALF])
def test_unusual_scales_in_large_tiles(shape, edge, precision):
    """X far below eps (its power of two at work) and far above, in tiles of
    128 and 256 with steps in pairs; a NaN fills the matrix."""
    T = torch()
    assert tile_edge([shape], precision) == edge
    T.manual_seed(9)
    x = T.randn(*shape, device="cuda")
    y = T.empty_like(x)
    table = lso.MatrixTable.from_rows([dict(x=x, y=y, rows=shape[0], cols=shape[1])])
    need = lso.orthogonalize_workspace_bytes(table, precision)
    ws = workspace(need)
    for f in (1e-30, 1e28):
        x.mul_(f)
        log(f"large tiles {shape} precision {precision} times {f}")
        lso.orthogonalize(table, ws, need, precision=precision)
        T.cuda.synchronize()
        want = ortho64_gpu(x)
        err = float((y.double() - want).norm() / want.norm())
        assert err <= tolerance(*shape, precision == FULL, False), (shape, f, err)
        x.div_(f)
    for value, ok in ((float("nan"), False), (0.0, True)):
        x.zero_() if ok else x[shape[0] - 1, 7].fill_(value)
        log(f"large tiles {shape} precision {precision} with {value}")
        lso.orthogonalize(table, ws, need, precision=precision)
        T.cuda.synchronize()
        assert bool((y == 0).all()) if ok else bool(y.isnan().all())
    assert bool((ws[need:] == CANARY).all())


# ------------------------------------------------------- large tiles, every form

@pytest.mark.parametrize("precision", [FULL, HALF])
@pytest.mark.parametrize("pad", [4, 3])     # rows in groups of four columns; columns one by one
@pytest.mark.parametrize("shapes,edge", [([(2100, 5100), (4100, 2000)], 128), ([(4100, 16100)], 256)])
def test_bf16_in_large_tiles(shapes, edge, pad, precision):
    """BF16 matrices with strides, in place of the FP32 ones without."""
    T = torch()
    assert tile_edge(shapes, precision) == edge
    T.manual_seed(4)
    xs = [T.randn(r, c + pad, device="cuda").bfloat16()[:, :c] for r, c in shapes]
    ys = [T.full((r, c + pad), 7.0, dtype=T.bfloat16, device="cuda") for r, c in shapes]
    table = lso.MatrixTable.from_rows(dict(x=x, y=y[:, :x.shape[1]], rows=x.shape[0], cols=x.shape[1]) for x, y in zip(xs, ys))
    need = lso.orthogonalize_workspace_bytes(table, precision)
    ws = workspace(need)
    log(f"BF16 in large tiles {shapes} pad {pad} precision {precision}")
    lso.orthogonalize(table, ws, need, precision=precision)
    T.cuda.synchronize()
    assert bool((ws[need:] == CANARY).all())
    for (r, c), x, y in zip(shapes, xs, ys):
        assert bool((y[:, c:] == 7.0).all())
        want = ortho64_gpu(x.contiguous())
        off = (y[:, :c].double() - want).abs()
        tol = tolerance(r, c, precision == FULL, False)
        norm = float(want.norm())
        assert float(off.norm()) <= (tol + 2.0**-8) * norm, (r, c, float(off.norm()) / norm)
        # an element: its rounding, and a few times its share of the rest
        assert bool((off <= 2.0**-8 * want.abs() + 12 * (1 + 2.0**-8) * tol * norm / math.sqrt(r * c)).all())


@pytest.mark.parametrize("shapes,edge,grad,weight,shift,precision", [
    ([(2100, 5100), (4100, 2000)], 128, "f32", True, 0, FULL),
    ([(2100, 5100), (4100, 2000)], 128, "bf16", False, 0, FULL),
    ([(2100, 5100), (4100, 2000)], 128, "bf16", True, 1, FULL),
    ([(2100, 5100), (4100, 2000)], 128, "bf16", True, 0, HALF),
    ([(4100, 16100)], 256, "bf16", True, 0, FULL),
    ([(4100, 16100)], 256, "f32", False, 1, FULL),
    ([(16100, 4100)], 256, "f32", True, 0, FULL),
    ([(16100, 4100)], 256, "bf16", True, 1, FULL),
    ([(16100, 4100)], 256, "bf16", True, 0, HALF),
])
def test_update_in_large_tiles(shapes, edge, grad, weight, shift, precision):
    """Two steps of the update of matrices as large as a model's, against its
    definition in 64 bits; the bounds are Block.check's.  shift 1: no array is
    aligned to more than its elements."""
    T = torch()
    assert tile_edge(shapes, precision) == edge
    T.manual_seed(6)
    lr, beta, decay, scale = 0.02, 0.9, 0.1, 1.5
    n = sum(r * c for r, c in shapes)

    def dev(values, dtype):
        t = T.full((n + shift + 1,), 77.0, dtype=dtype, device="cuda")
        t[shift:shift + n] = values
        return t
    spikes = T.cat([(T.outer(T.randn(r, device="cuda"), T.randn(c, device="cuda")) * 4e-3).flatten() for r, c in shapes])
    master, m = dev(T.randn(n, device="cuda") * 0.02, T.float32), dev(T.randn(n, device="cuda") * 1e-3 + spikes, T.float32)
    g = dev(T.randn(n, device="cuda") * 1e-3 + spikes, T.float32 if grad == "f32" else T.bfloat16)
    w = dev(T.zeros(n, device="cuda"), T.bfloat16) if weight else None
    del spikes
    rows, at = [], shift
    for r, c in shapes:
        rows.append(dict(rows=r, cols=c, master=master[at:at + r * c], m=m[at:at + r * c], grad=g[at:at + r * c],
                         weight=w[at:at + r * c] if weight else None, lr=lr, beta=beta, weight_decay=decay, scale=scale))
        at += r * c
    table = lso.MuonTable.from_rows(rows)
    need = lso.muon_workspace_bytes(table, precision)
    ws = workspace(need)
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    b, c1, keep, step = f32(beta), f32(1 - beta), f32(1 - lr * decay), f32(-lr * scale)
    for k in range(2):
        own = slice(shift, shift + n)
        m0, p0, g64 = m[own].double(), master[own].double(), g[own].double()
        log(f"update in large tiles {shapes} grad {grad} weight {weight} shift {shift} precision {precision} step {k}")
        lso.muon_step(table, ws, need, precision=precision)
        T.cuda.synchronize()
        want_m = b * m0 + c1 * g64
        assert bool(((m[own].double() - want_m).abs() <= 2.0**-23 * ((b * m0).abs() + (c1 * g64).abs()) + 1e-45).all())
        u = b * want_m + c1 * g64
        del m0, want_m, g64
        at = 0
        for r, c in shapes:
            part = slice(at, at + r * c)
            y = ortho64_gpu(u[part].view(r, c)).flatten()
            want = keep * p0[part] + step * y
            tol = tolerance(r, c, precision == FULL, False) + 115 * 2.0**-22
            off = 12 * tol * float(y.norm()) / math.sqrt(r * c) + 2.0**-23 * float(y.abs().max())
            bound = 2.0**-23 * ((keep * p0[part]).abs() + (step * y).abs()) + abs(step) * off
            got = master[own][part].double()
            assert bool(((got - want).abs() <= bound).all()), (r, c, float(((got - want).abs() / bound).max()))
            # as a whole: what the orthogonalisation may be off
            err = float((got - want).norm())
            assert err <= abs(step) * tol * float(y.norm()) + 2.0**-23 * float((keep * p0[part]).norm()), (r, c, err)
            at += r * c
            del y, want, bound, got
        if weight:
            assert T.equal(w[own], master[own].bfloat16())
        for t in (master, m, g) + ((w,) if weight else ()):
            assert float(t[shift + n]) == 77.0 and bool((t[:shift] == 77.0).all()), "written beside an array"
        assert bool((ws[need:] == CANARY).all())


# ---------------------------------------------------------------- long tables

LONG = [(4, 40 + i % 90) for i in range(290)] + [(70, 80 + i % 7) for i in range(40)] + [(100 + i, 66) for i in range(6)]


@pytest.mark.parametrize("shapes", [LONG, LONG[:200] + LONG[-46:]])
def test_long_tables_with_general_matrices(shapes):
    """Tables that take one launch and more to write, their last entries
    general-path matrices; eagerly and in a graph."""
    assert len(LONG) > 314 and all(general(s) for s in LONG[-46:]) and not general(LONG[0])
    T = torch()
    eager, graphed = Block(shapes, "f32", True, seed=90, lr=0.1), Block(shapes, "f32", True, seed=90, lr=0.1)
    need = lso.muon_workspace_bytes(eager.table)
    ws = [workspace(need), workspace(need)]
    log(f"{len(shapes)} matrices eager")
    run_muon(eager)
    eager.check(what="eager")
    log(f"{len(shapes)} matrices captured")
    g = T.cuda.CUDAGraph()
    with T.cuda.graph(g):
        lso.muon_step(graphed.table, ws[1], need)
    for k in range(3):
        g.replay()
        T.cuda.synchronize()
        if k > 0:
            lso.muon_step(eager.table, ws[0], need)
            T.cuda.synchronize()
        assert T.equal(eager.master, graphed.master) and T.equal(eager.m, graphed.m) and T.equal(eager.w, graphed.w), f"replay {k}"
