"""embed_lookup and embed_grad on the GPU against their definitions in 64 bits.

Tolerances.  A looked-up element is one FP32 product, rounded once more to
BF16 where asked: at most 2^-24 and 2^-8 of its size (half a step: FP32
neighbours in [1, 2) are 2^-23 apart, BF16 ones 2^-7).  A gradient element is a sum of c
values in FP32, at most c roundings of 2^-24 of the sum of the values'
sizes, then the scaling (2^-24), an addition (2^-24 of the result and of what
was there) and the rounding to the table's type."""
import ctypes

import numpy as np
import pytest

import layer_streamed_optimizer_amd as lso
from layer_streamed_optimizer_amd import _native

from gpu_util import log, torch

pytestmark = pytest.mark.gpu

DT = {"f32": "float32", "bf16": "bfloat16", "i32": "int32", "i64": "int64"}


def td(name):
    return getattr(torch(), DT[name])


def tokens(n, vocab, seed, kind="zipf"):
    rng = np.random.default_rng(seed)
    if kind == "same":
        return np.full(n, vocab // 2, np.int64)
    if kind == "ramp":
        return (np.arange(n, dtype=np.int64) * 7919) % vocab
    if kind == "padding":
        return np.where(np.arange(n) % 2 == 0, -1, vocab).astype(np.int64)
    t = np.minimum(rng.zipf(1.3, n) - 1, vocab + 3)   # a few beyond the table
    t[rng.random(n) < 0.05] = -1
    return t.astype(np.int64)


def rounding(dt):
    return 2.0**-8 if dt == "bf16" else 2.0**-24


class Strided:
    """rows x cols with `pad` elements between rows, canaries in them and around."""

    def __init__(self, rows, cols, dt, pad=0, shift=0, fill=None):
        T = torch()
        self.rows, self.cols, self.ld = rows, cols, cols + pad
        self.raw = T.full((rows * self.ld + 32 + shift,), 55.0, dtype=td(dt), device="cuda")
        self.t = self.raw[16 + shift:16 + shift + rows * self.ld].view(rows, self.ld)[:, :cols]
        if fill is not None:
            self.t.copy_(T.from_numpy(fill))

    def host(self):
        return self.t.float().cpu().numpy().astype(np.float64)

    def check_canaries(self):
        T = torch()
        c = self.raw.clone()
        off = self.t.storage_offset()
        c[off:off + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] = 55.0
        assert bool((c == 55.0).all()), "written outside"


def workspace(nbytes):
    ws = torch().full((nbytes + 256,), 0xFF, dtype=torch().uint8, device="cuda")
    return ws


@pytest.mark.parametrize("index", ["i32", "i64"])
@pytest.mark.parametrize("table,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("n,vocab,width,pad", [(1, 10, 8, 0), (1, 1, 1, 0), (5, 33, 7, 3), (64, 1000, 4096, 0), (300, 77, 513, 0),
                                                (257, 500, 1000, 8), (3000, 900, 72, 4), (20000, 3000, 520, 0)])
def test_lookup(index, table, out, n, vocab, width, pad):
    log(f"lookup {index} {table}->{out} n {n} vocab {vocab} width {width} pad {pad}")
    rng = np.random.default_rng(n + width)
    w = Strided(vocab, width, table, pad, fill=rng.standard_normal((vocab, width)).astype(np.float32))
    o = Strided(n, width, out, pad)
    t = tokens(n, vocab, n)
    scale = 1.7
    lso.embed_lookup(torch().from_numpy(t).to(td(index)).cuda(), w.t, o.t, scale=scale)
    torch().cuda.synchronize()
    ok = (t >= 0) & (t < vocab)
    want = np.where(ok[:, None], w.host()[np.clip(t, 0, vocab - 1)] * np.float64(np.float32(scale)), 0.0)
    got = o.host()
    assert np.all(np.abs(got - want) <= (2.0**-24 + rounding(out)) * np.abs(want))
    o.check_canaries()


def grad_reference(t, dy, vocab, scale, old=None):
    """(value, sum of sizes, count) in 64 bits."""
    out = np.zeros((vocab, dy.shape[1]))
    size, count = np.zeros_like(out), np.zeros(vocab)
    ok = (t >= 0) & (t < vocab)
    np.add.at(out, t[ok], dy[ok])
    np.add.at(size, t[ok], np.abs(dy[ok]))
    np.add.at(count, t[ok], 1)
    s = np.float64(np.float32(scale))
    out, size = out * s, size * abs(s)
    if old is not None:
        out = out + old
        size = size + np.abs(old)
    return out, size, count


def run_grad(t, dy, grad, index="i64", scale=1.0, accumulate=False):
    n, vocab, width = len(t), grad.t.shape[0], grad.t.shape[1]
    need = lso.embed_grad_workspace_bytes(n, vocab, width)
    ws = workspace(need)
    lso.embed_grad(torch().from_numpy(t).to(td(index)).cuda(), dy.t, grad.t, ws, need, scale=scale, accumulate=accumulate)
    torch().cuda.synchronize()
    assert bool((ws[need:] == 0xFF).all()), "written behind the workspace"
    grad.check_canaries()


def check_grad(t, dy, grad, before, grad_dt, scale, accumulate):
    old = before if accumulate else None
    want, size, count = grad_reference(t, dy.host(), grad.t.shape[0], scale, old)
    got = grad.host()
    tol = (count[:, None] + 3) * 2.0**-24 * size + rounding(grad_dt) * np.abs(want)
    bad = np.abs(got - want) > tol
    assert not bad.any(), f"{bad.sum()} elements, first row {np.argwhere(bad)[0]}, off by {np.max(np.abs(got - want) / np.maximum(tol, 1e-300)):.3g}"
    if accumulate:
        untouched = count == 0
        assert np.array_equal(got[untouched], before[untouched])   # bit for bit, signed zeros aside
    else:
        assert not got[count == 0].any()


GRADS = [
    # n, vocab, width, pad, kind
    (0, 9, 16, 0, "zipf"), (1, 1, 1, 0, "same"), (1, 50, 8, 0, "same"), (31, 40, 9, 2, "zipf"), (32, 40, 16, 0, "same"),
    (33, 40, 16, 0, "same"), (34, 5, 24, 8, "ramp"), (64, 3, 512, 0, "ramp"), (65, 200, 8, 0, "padding"), (257, 1023, 130, 0, "zipf"),
    (1000, 1024, 520, 0, "zipf"), (1000, 32000, 64, 0, "zipf"), (2049, 7, 40, 0, "ramp"), (4096, 128, 1032, 0, "same"),
    (5000, 70000, 24, 0, "ramp"), (9001, 300, 65, 1, "zipf"), (20000, 1 << 20, 8, 0, "zipf"), (140000, 1000, 16, 0, "zipf"),
]


@pytest.mark.parametrize("n,vocab,width,pad,kind", GRADS)
@pytest.mark.parametrize("dy_dt,grad_dt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_gradient(n, vocab, width, pad, kind, dy_dt, grad_dt):
    rng = np.random.default_rng(n + vocab)
    t = tokens(n, vocab, n + 1, kind)
    dy = Strided(n, width, dy_dt, pad, fill=rng.standard_normal((n, width)).astype(np.float32))
    for accumulate in (False, True):
        start = rng.standard_normal((vocab, width)).astype(np.float32) if accumulate else None
        grad = Strided(vocab, width, grad_dt, pad, fill=start)
        before = grad.host()
        index = "i32" if accumulate else "i64"
        log(f"grad n {n} vocab {vocab} width {width} pad {pad} {kind} {dy_dt}->{grad_dt} add {accumulate}")
        run_grad(t, dy, grad, index, scale=0.75, accumulate=accumulate)
        check_grad(t, dy, grad, before, grad_dt, 0.75, accumulate)


def test_gradient_is_the_derivative_of_the_lookup():
    """<lookup(W + h D) - lookup(W - h D), dy> / 2h = <grad, D>: both are
    linear in W, so the difference quotient is exact but for roundings."""
    n, vocab, width, scale = 200, 37, 24, 3.0
    rng = np.random.default_rng(8)
    t = tokens(n, vocab, 2)
    dyh = rng.integers(-8, 9, (n, width)).astype(np.float32)     # small whole numbers: every sum is exact
    d = rng.integers(-8, 9, (vocab, width)).astype(np.float32)
    w = rng.integers(-8, 9, (vocab, width)).astype(np.float32)
    dt = torch().from_numpy(t).cuda()
    outs = []
    log("lookup and gradient")
    for s in (1, -1):
        o = Strided(n, width, "f32")
        lso.embed_lookup(dt, Strided(vocab, width, "f32", fill=w + s * d).t, o.t, scale=scale)
        outs.append(o.host())
    grad, dy = Strided(vocab, width, "f32"), Strided(n, width, "f32", fill=dyh)
    run_grad(t, dy, grad, scale=scale)
    assert ((outs[0] - outs[1]) / 2 * dyh).sum() == (grad.host() * d).sum()


def test_gradient_ignores_what_padding_holds_and_repeats_bit_for_bit():
    n, vocab, width = 5000, 60, 264
    rng = np.random.default_rng(4)
    t = tokens(n, vocab, 5)
    fill = rng.standard_normal((n, width)).astype(np.float32)
    fill[(t < 0) | (t >= vocab)] = np.nan
    dy = Strided(n, width, "f32", fill=fill)
    a, b = Strided(vocab, width, "f32"), Strided(vocab, width, "f32")
    log("gradient with NaN in padding")
    run_grad(t, dy, a)
    run_grad(t, dy, b)
    assert np.isfinite(a.host()).all() and np.array_equal(a.host(), b.host())


def test_two_gradients_at_once_on_two_streams():
    T = torch()
    n, vocab, width = 9000, 400, 512
    rng = np.random.default_rng(6)
    calls = []
    for k in range(2):
        t = tokens(n, vocab, 40 + k)
        dy = Strided(n, width, "bf16", fill=rng.standard_normal((n, width)).astype(np.float32))
        one, two = Strided(vocab, width, "f32"), Strided(vocab, width, "f32")
        run_grad(t, dy, one)
        need = lso.embed_grad_workspace_bytes(n, vocab, width)
        calls.append((T.from_numpy(t).cuda(), dy, one, two, workspace(need), need, T.cuda.Stream()))
    T.cuda.synchronize()
    log("two gradients at once")
    for _ in range(3):
        for t, dy, _, two, ws, need, s in calls:
            lso.embed_grad(t, dy.t, two.t, ws, need, stream=s)
    T.cuda.synchronize()
    for _, _, one, two, _, _, _ in calls:
        assert T.equal(one.t, two.t)


def test_wide_token_values_are_padding_not_wrapped():
    t = np.array([1, (1 << 32) + 1, -(1 << 32) + 1, (1 << 62), 2], np.int64)
    fill = np.arange(1, 41, dtype=np.float32).reshape(5, 8)
    dy, grad = Strided(5, 8, "f32", fill=fill), Strided(4, 8, "f32")
    log("wide tokens")
    run_grad(t, dy, grad)
    want = np.zeros((4, 8))
    want[1], want[2] = fill[0], fill[4]
    assert np.array_equal(grad.host(), want)
    w, o = Strided(4, 8, "f32", fill=fill[:4]), Strided(5, 8, "f32")
    lso.embed_lookup(torch().from_numpy(t).cuda(), w.t, o.t)
    got = o.host()
    assert np.array_equal(got[0], fill[1]) and np.array_equal(got[4], fill[2]) and not got[1:4].any()


def test_offsets_beyond_32_bits():
    """A table of more than 2^32 elements: the last rows are found."""
    T = torch()
    vocab, width = 1_100_000, 4096   # 4.5e9 elements, 9 GB in BF16
    w = T.zeros(vocab, width, dtype=T.bfloat16, device="cuda")
    w[vocab - 1] = 3.0
    t = T.tensor([vocab - 1, 0, vocab, vocab - 1], device="cuda")
    o = T.full((4, width), 9.0, device="cuda")
    log("lookup in a large table")
    lso.embed_lookup(t, w, o, scale=2.0)
    assert o[:, 0].tolist() == [6.0, 0.0, 0.0, 6.0] and bool((o == o[:, :1]).all())
    need = lso.embed_grad_workspace_bytes(4, vocab, width)
    w.fill_(1.0)
    log("gradient of a large table")
    lso.embed_grad(t, o, w, workspace(need), need)
    T.cuda.synchronize()
    assert float(w[vocab - 1].float().min()) == 12.0 == float(w[vocab - 1].float().max())
    assert not w[vocab - 2].any() and not w[1].any() and not w[0].any()


def test_lookup_update_gradient_in_one_graph():
    """A training step's use of the table: lookup of the BF16 weights, the
    gradient into the block's gradient array, the Adam update of the block;
    captured once, replayed on new batches, equal to the eager steps."""
    T = torch()
    n, vocab, width = 300, 128, 64

    def make():
        d = dict(master=T.linspace(-1, 1, vocab * width, device="cuda"), m=T.zeros(vocab * width, device="cuda"),
                 v=T.zeros(vocab * width, device="cuda"), grad=T.zeros(vocab, width, dtype=T.bfloat16, device="cuda"),
                 weight=T.linspace(-1, 1, vocab * width, device="cuda").bfloat16())
        s = dict(d=d, tokens=T.zeros(n, dtype=T.int64, device="cuda"), out=T.zeros(n, width, dtype=T.bfloat16, device="cuda"))
        s["need"] = lso.embed_grad_workspace_bytes(n, vocab, width)
        s["ws"] = workspace(s["need"])
        s["table"] = lso.BlockTable.from_rows([dict(n=vocab * width, t=1, lr=0.1, **d)])
        return s

    def step(s):
        lso.embed_lookup(s["tokens"], s["d"]["weight"].view(vocab, width), s["out"], scale=2.0)
        lso.embed_grad(s["tokens"], s["out"], s["d"]["grad"], s["ws"], s["need"], scale=2.0)
        lso.adam_step_noalloc(s["table"])
    a, b = make(), make()
    log("embedding step eager")
    step(a)
    T.cuda.synchronize()
    a = make()
    log("embedding step captured")
    g = T.cuda.CUDAGraph()
    with T.cuda.graph(g):
        step(b)
    for k in range(4):
        for s in (a, b):
            s["tokens"].copy_(T.from_numpy(tokens(n, vocab, k)))
        g.replay()
        T.cuda.synchronize()
        step(a)
        T.cuda.synchronize()
        assert T.equal(a["out"], b["out"])
        for key in ("grad", "weight", "master", "m", "v"):
            assert T.equal(a["d"][key], b["d"][key]), (k, key)
    assert a["d"]["grad"].any()


@pytest.mark.parametrize("grad_dt", ["bf16", "f32"])
def test_producer_in_the_layer_stream(grad_dt):
    """An embedding table streamed from host memory with its gradient made by
    the library's own producer, beside a layer of another producer: the same
    state as the resident update with embed_grad's gradient."""
    import synth
    from layer_streamed_optimizer_amd import configs
    T = torch()
    n, vocab, width = 500, 70, 40
    code = lso.LSO_DT_BF16 if grad_dt == "bf16" else lso.LSO_DT_F32
    sizes = [3000, vocab * width]
    lay = [configs.host_layer_layout(k) for k in sizes]
    t = tokens(n, vocab, 3)
    dt = T.from_numpy(t).cuda()
    dy = T.randn(n, width, device="cuda") * 1e-2
    need = lso.embed_grad_workspace_bytes(n, vocab, width)
    ws = workspace(need)
    other, Params = synth.grad_callback()
    prm = Params(seed=synth.SEED, stream=90, purpose=synth.PURPOSE_GRAD, step=1, scale=synth.scale_for(1e-3), block_base=0)
    if grad_dt == "f32":
        other_ptr, other_user, layers = 0, 0, [1]     # the other producer writes BF16
    else:
        other_ptr, other_user, layers = other, ctypes.addressof(prm), [0, 1]
    p = lso.EmbedProducer(dt, dy, vocab, width, ws, need, embed_layer=1, grad_dtype=code, scale=1.5, other=other_ptr,
                          other_user=other_user)
    ls = lso.LayerStream(max(x[3] for x in lay), max(sizes), p.fn, p.user)
    L = lso.LayerStream.layers(2)
    bufs = []
    for i, k in enumerate(sizes):
        om, omm, ov, nbytes = lay[i]
        hb = lso.host_alloc(nbytes)
        hb.view(np.uint8)[:] = 0
        hb.view(np.float32, om, k)[:] = np.linspace(-1, 1, k, dtype=np.float32)
        bufs.append(hb)
        L[i]["host_base"], L[i]["bytes"], L[i]["n"] = hb.ptr, nbytes, k if i in layers else 0
        L[i]["off_master"], L[i]["off_m"], L[i]["off_v"] = om, omm, ov
        L[i]["t"], L[i]["lr"], L[i]["beta1"], L[i]["beta2"], L[i]["eps"] = 1, 1e-2, 0.9, 0.999, 1e-8
        L[i]["grad_dtype"] = code
    log(f"layer stream with the embedding producer, {grad_dt}")
    ls.stream_layers(L)
    # resident: the same gradient, the same update
    grad = T.zeros(vocab, width, dtype=td(grad_dt), device="cuda")
    lso.embed_grad(dt, dy, grad, ws, need, scale=1.5)
    st = dict(master=T.from_numpy(np.linspace(-1, 1, sizes[1], dtype=np.float32)).cuda(), m=T.zeros(sizes[1], device="cuda"),
              v=T.zeros(sizes[1], device="cuda"))
    lso.adam_step(lso.BlockTable.from_rows([dict(n=sizes[1], grad=grad, t=1, lr=1e-2, grad_dtype=code, **st)]))
    T.cuda.synchronize()
    for q, off in zip(("master", "m", "v"), lay[1][:3]):
        assert np.array_equal(bufs[1].view(np.float32, off, sizes[1]), st[q].cpu().numpy()), q
    if 0 in layers:
        assert bufs[0].view(np.float32, lay[0][1], sizes[0]).any()
    ls.close()
    for hb in bufs:
        hb.close()


def test_gradient_refuses_a_workspace_tensor_that_is_too_small():
    """(Refused before anything is enqueued.)"""
    T = torch()
    t, dy, grad = T.zeros(100, dtype=T.int64, device="cuda"), T.zeros(100, 16, device="cuda"), T.full((8, 16), 3.0, device="cuda")
    need = lso.embed_grad_workspace_bytes(100, 8, 16)
    log("gradient with workspaces that are refused")
    for ws in (T.empty(need - 1, dtype=T.uint8, device="cuda"), T.empty(need, dtype=T.uint8), T.empty(2 * need, dtype=T.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            lso.embed_grad(t, dy, grad, ws, need)
    T.cuda.synchronize()
    assert bool((grad == 3.0).all())


def test_producer_waits_for_the_batch_it_is_given():
    """A batch that is still being written when the producer gets it: the layer
    stream's update uses what it ends as."""
    from layer_streamed_optimizer_amd import configs
    T = torch()
    n, vocab, width = 300, 50, 64
    om, omm, ov, nbytes = configs.host_layer_layout(vocab * width)
    t = T.from_numpy(tokens(n, vocab, 3)).cuda()
    first, dy = T.ones(n, width, device="cuda"), T.zeros(n, width, device="cuda")
    need = lso.embed_grad_workspace_bytes(n, vocab, width)
    ws = workspace(need)
    p = lso.EmbedProducer(t, first, vocab, width, ws, need, grad_dtype=lso.LSO_DT_F32)
    ls = lso.LayerStream(nbytes, vocab * width, p.fn, p.user)
    hb = lso.host_alloc(nbytes)
    hb.view(np.uint8)[:] = 0
    L = lso.LayerStream.layers(1)
    L[0]["host_base"], L[0]["bytes"], L[0]["n"] = hb.ptr, nbytes, vocab * width
    L[0]["off_master"], L[0]["off_m"], L[0]["off_v"] = om, omm, ov
    L[0]["t"], L[0]["lr"], L[0]["beta1"], L[0]["beta2"], L[0]["eps"] = 1, 1e-2, 0.9, 0.999, 1e-8
    L[0]["grad_dtype"] = lso.LSO_DT_F32
    a = T.randn(4096, 4096, device="cuda")
    T.cuda.synchronize()
    log("producer with a batch that is being written")
    with T.cuda.stream(T.cuda.Stream()):
        for _ in range(8):
            a = a @ a * 1e-2                 # some milliseconds of work before the batch is there
        dy.fill_(2.0)
        p.set_batch(t, dy)
        ls.stream_layers(L)
    want = np.zeros(vocab)
    host = t.cpu().numpy()
    np.add.at(want, host[(host >= 0) & (host < vocab)], 2.0)
    m = hb.view(np.float32, omm, vocab * width).reshape(vocab, width).astype(np.float64)
    # m' = (1 - beta1) g: g is exact, the constant and the product are rounded
    assert np.all(np.abs(m - 0.1 * want[:, None]) <= 2.001 * 2.0**-24 * 0.1 * want[:, None])
    ls.close()
    hb.close()


def test_an_error_left_by_other_work_stays_there():
    """An error that other code of the thread has not collected: the calls
    neither report it nor take it away."""
    from test_gpu_matrix import Block, Mats
    T, lib = torch(), _native.lib()
    n, vocab, width = 5000, 40, 64
    t = T.from_numpy(tokens(n, vocab, 1)).cuda()
    w, o = Strided(vocab, width, "f32", fill=np.ones((vocab, width), np.float32)), Strided(n, width, "f32")
    need = lso.embed_grad_workspace_bytes(n, vocab, width)
    ws = workspace(need)
    e = _native.LsoEmbed(t.data_ptr(), n, w.t.data_ptr(), vocab, width, width, o.t.data_ptr(), width, 4, 1, 1, 0, 1.0)
    m, b = Mats([(9, 30), (70, 90)], seed=1), Block([(9, 30), (70, 90)], "f32", False, seed=1)
    mw = max(lso.orthogonalize_workspace_bytes(m.table), lso.muon_workspace_bytes(b.table))
    mws = workspace(mw)
    T.cuda.synchronize()
    calls = [lambda: lib.lso_embed_lookup(ctypes.byref(e), None), lambda: lib.lso_embed_grad(ctypes.byref(e), ws.data_ptr(), need, None),
             lambda: lib.lso_orthogonalize(m.table.ptr, 2, None, mws.data_ptr(), mw, None),
             lambda: lib.lso_muon_step(b.table.ptr, 2, None, mws.data_ptr(), mw, None)]
    log("calls beside an uncollected error")
    for call in calls:
        assert call() == 0               # (and the code objects are loaded)
    lib.hipGetLastError()
    seen = []
    for call in calls:
        left = lib.hipSetDevice(ctypes.c_int(1 << 20))    # no such device: a host-side refusal
        status = call()
        seen.append((left != 0, status, lib.hipGetLastError() == left, lib.hipGetLastError()))
    T.cuda.synchronize()
    assert seen == [(True, 0, True, 0)] * 4


L2_BYTES = 32 << 20      # rows of more than this are read, or written, past the caches


def grad_on_device(t, dy, vocab, scale, old):
    """grad_reference on the device: (value, sum of sizes, count) in 64 bits."""
    T = torch()
    real = (t >= 0) & (t < vocab)
    ids, rows = t[real].long(), dy[real].double()
    out = T.zeros(vocab, dy.shape[1], dtype=T.float64, device="cuda")
    size, count = T.zeros_like(out), T.bincount(ids, minlength=vocab).double()
    out.index_add_(0, ids, rows)
    size.index_add_(0, ids, rows.abs())
    s = float(np.float32(scale))
    out, size = out * s, size * abs(s)
    if old is not None:
        out, size = out + old, size + old.abs()
    return out, size, count


@pytest.mark.parametrize("n,vocab,width,pad,kind", [(20000, 3000, 1024, 0, "zipf"), (9000, 20000, 2048, 8, "zipf"),
                                                    (33000, 32000, 520, 0, "ramp"), (40000, 17, 424, 0, "ramp"), (17000, 2, 1032, 0, "same")])
@pytest.mark.parametrize("dy_dt,grad_dt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_gradient_of_rows_beyond_the_caches(n, vocab, width, pad, kind, dy_dt, grad_dt):
    """Long and short runs, padding and empty rows among them."""
    T = torch()
    assert n * width * (2 if dy_dt == "bf16" else 4) > L2_BYTES and width % 8 == 0 and pad % 8 == 0
    T.manual_seed(n)
    t = T.from_numpy(tokens(n, vocab, n + 2, kind))
    if kind != "zipf":
        t[::9] = -1
    t = t.cuda()
    dy = Strided(n, width, dy_dt, pad)
    dy.t.copy_(T.randn(n, width, device="cuda"))
    need = lso.embed_grad_workspace_bytes(n, vocab, width)
    for accumulate in (False, True):
        grad = Strided(vocab, width, grad_dt, pad)
        if accumulate:
            grad.t.copy_(T.randn(vocab, width, device="cuda"))
        before = grad.t.clone()
        ws = workspace(need)
        log(f"grad beyond the caches n {n} vocab {vocab} width {width} pad {pad} {kind} {dy_dt}->{grad_dt} add {accumulate}")
        lso.embed_grad(t.int() if accumulate else t, dy.t, grad.t, ws, need, scale=0.75, accumulate=accumulate)
        T.cuda.synchronize()
        assert bool((ws[need:] == 0xFF).all()), "written behind the workspace"
        grad.check_canaries()
        want, size, count = grad_on_device(t, dy.t, vocab, 0.75, before.double() if accumulate else None)
        tol = (count[:, None] + 3) * 2.0**-24 * size + rounding(grad_dt) * want.abs()
        assert bool(((grad.t.double() - want).abs() <= tol).all())
        empty = count == 0
        assert T.equal(grad.t[empty], before[empty]) if accumulate else not bool(grad.t[empty].any())


@pytest.mark.parametrize("table", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_lookup_of_rows_beyond_the_caches(table, out):
    T = torch()
    n, vocab, width = 20000, 3000, 1032
    assert n * width * (2 if out == "bf16" else 4) > L2_BYTES
    t = T.from_numpy(tokens(n, vocab, 4)).cuda()
    w, o = Strided(vocab, width, table, 8), Strided(n, width, out, 8)
    w.t.copy_(T.randn(vocab, width, device="cuda"))
    log(f"lookup beyond the caches {table}->{out}")
    lso.embed_lookup(t, w.t, o.t, scale=1.7)
    T.cuda.synchronize()
    real = (t >= 0) & (t < vocab)
    want = T.where(real[:, None], w.t.double()[t.clamp(0, vocab - 1)] * float(np.float32(1.7)), 0.0)
    assert bool(((o.t.double() - want).abs() <= (2.0**-24 + rounding(out)) * want.abs()).all())
    o.check_canaries()
