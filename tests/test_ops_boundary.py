"""The boundary of include/lso_ops.h on the CPU: symbols, layouts, constants
and every refusal of its calls.  Addresses are made up: a refused call
touches no memory, and no call here is a valid one."""
import ctypes
import os
import re
import subprocess
from unittest import mock

import numpy as np
import pytest

import layer_streamed_optimizer_amd as lso
from layer_streamed_optimizer_amd import _native, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lso_ops.h")
A = 1 << 32   # fake device addresses
WS = 1 << 40
BIG = 1 << 36
INVALID, ALIGN, DTYPE, OVERLAP = 1, 2, 3, 4


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(lso_[a-z0-9_]+)\s*\(", text))
    assert names == set(_native.OPS_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", _native._build.lib_path()], capture_output=True, text=True,
                         check=True).stdout
    assert names <= set(re.findall(r"\sT\s+(lso_\w+)", out))


def test_struct_layouts_and_constants_match_the_header(tmp_path):
    structs = {"lso_ns_params": _native.LsoNsParams, "lso_matrix": _native.LsoMatrix, "lso_muon_block": _native.LsoMuonBlock,
               "lso_embed": _native.LsoEmbed, "lso_embed_producer_args": _native.LsoEmbedProducerArgs}
    consts = ("LSO_NS_AUTO", "LSO_NS_FULL", "LSO_NS_HALF", "LSO_NS_SMALL_SIDE", "LSO_NS_MAX_STEPS", "LSO_MUON_NESTEROV",
              "LSO_DT_I32", "LSO_DT_I64", "LSO_EMBED_ADD")
    lines = [f'printf("{s} %zu\\n", sizeof({s}));' for s in structs]
    lines += [f'printf("{s}.{f} %zu\\n", offsetof({s}, {f}));' for s, c in structs.items() for f, _ in c._fields_]
    lines += [f'printf("{c} %u\\n", (unsigned){c});' for c in consts]
    src = tmp_path / "l.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"lso_ops.h\"\nint main(void) {\n" + "\n".join(lines) +
                   "\nreturn 0; }\n")
    exe = str(tmp_path / "l")
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe])
    got = {k: int(v) for k, v in (line.split() for line in subprocess.run([exe], capture_output=True, text=True).stdout.split("\n") if line)}
    for s, c in structs.items():
        assert got[s] == ctypes.sizeof(c), s
        for f, _ in c._fields_:
            assert got[f"{s}.{f}"] == getattr(c, f).offset, (s, f)
    for c in consts:
        assert got[c] == getattr(_native, c), c


# ------------------------------------------------------------------ matrices

def mat(k=0, **kw):
    d = dict(x=A + k * (1 << 28), y=A + (1 << 27) + k * (1 << 28), rows=100, cols=200)
    d.update(kw)
    return d


def ortho(rows, ws=WS, nbytes=BIG, **kw):
    with pytest.raises(lso.LsoError) as e:
        lso.orthogonalize(lso.MatrixTable.from_rows(rows), ws, nbytes, stream=0, **kw)
    return e.value.status


@pytest.mark.parametrize("rows,code", [
    ([mat(x=0)], INVALID), ([mat(y=0)], INVALID), ([mat(ld_x=199)], INVALID), ([mat(ld_y=199)], INVALID),
    ([mat(ld_x=1 << 31)], INVALID), ([mat(rows=1 << 31)], INVALID), ([mat(cols=1 << 32)], INVALID),
    ([mat(x=A + 2)], ALIGN), ([mat(x=A + 1, x_dtype=2)], ALIGN), ([mat(y=A + (1 << 27) + 2)], ALIGN),
    ([mat(x_dtype=0)], DTYPE), ([mat(y_dtype=3)], DTYPE),
    ([mat(y=A + 4)], OVERLAP),                                   # y inside x
    ([mat(y=A, y_dtype=2)], OVERLAP), ([mat(y=A, ld_y=201)], OVERLAP),   # in place only with x's type and stride
    ([mat(), mat(1, y=A + (1 << 27) + 400)], OVERLAP),           # two results
    ([mat(), mat(1, x=A + (1 << 27))], OVERLAP),                 # a result and another's input
    ([mat(rows=1 << 30, cols=1 << 30)], INVALID),                # more elements than can be addressed
])
def test_orthogonalize_refuses(rows, code):
    assert ortho(rows) == code
    assert lso.ops._native.lib().lso_last_error()


def test_orthogonalize_refuses_workspaces():
    tab = lso.MatrixTable.from_rows([mat(), mat(1, rows=8)])
    need = lso.orthogonalize_workspace_bytes(tab)
    assert need > 0
    assert ortho([mat(), mat(1, rows=8)], ws=None) == INVALID
    assert ortho([mat(), mat(1, rows=8)], ws=WS + 8) == ALIGN
    assert ortho([mat(), mat(1, rows=8)], nbytes=need - 1) == INVALID
    assert ortho([mat(), mat(1, rows=8)], ws=A - 16) == OVERLAP
    # full precision holds more than half precision does
    assert lso.orthogonalize_workspace_bytes(tab, lso.LSO_NS_FULL) > lso.orthogonalize_workspace_bytes(tab, lso.LSO_NS_HALF)


@pytest.mark.parametrize("kw", [
    dict(steps=0), dict(steps=17), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(precision=3),
    dict(coefficients=(float("nan"), 0, 0)), dict(coefficients=(16.0, 0, 0)), dict(coefficients=(2.0, 0.0, 0.0), steps=5),
    dict(coefficients=(3.0, 3.0, 3.0)), dict(coefficients=(0.0, -100.0, 100.0), steps=1),
])
def test_orthogonalize_refuses_parameters(kw):
    assert ortho([mat()], **kw) == INVALID


def test_coefficient_shapes():
    tab = lso.MatrixTable.from_rows([mat()])
    with pytest.raises(ValueError):
        lso.orthogonalize(tab, WS, BIG, steps=3, coefficients=[(1, 0, 0)] * 2, stream=0)


def test_empty_matrix_calls_are_no_ops():
    lso.orthogonalize(lso.MatrixTable(0), None, 0, stream=0)
    lso.orthogonalize(lso.MatrixTable.from_rows([mat(rows=0, x=0, y=0), mat(cols=0, x=0, y=0)]), None, 0, stream=0)
    lso.muon_step(lso.MuonTable.from_rows([block(rows=0, master=0, m=0, grad=0)]), None, 0, stream=0)
    assert lso.orthogonalize_workspace_bytes(lso.MatrixTable(0)) == 0


def block(k=0, **kw):
    base = A + k * (1 << 28)
    d = dict(rows=64, cols=96, master=base, m=base + (1 << 20), grad=base + (2 << 20), weight=base + (3 << 20))
    d.update(kw)
    return d


def muon(rows, edit=None, ws=WS, nbytes=BIG):
    tab = lso.MuonTable.from_rows(rows)
    if edit:
        edit(tab.arr)
    with pytest.raises(lso.LsoError) as e:
        lso.muon_step(tab, ws, nbytes, stream=0)
    return e.value.status


@pytest.mark.parametrize("rows,code", [
    ([block(master=0)], INVALID), ([block(m=0)], INVALID), ([block(grad=0)], INVALID), ([block(weight=0)], INVALID),
    ([block(lr=float("inf"))], INVALID), ([block(beta=1.0)], INVALID), ([block(beta=-0.1)], INVALID),
    ([block(weight_decay=float("nan"))], INVALID), ([block(scale=float("inf"))], INVALID), ([block(lr=1e30, scale=1e30)], INVALID),
    ([block(grad_dtype=0)], DTYPE), ([block(grad_dtype=3)], DTYPE), ([block(master=A + 2)], ALIGN), ([block(weight=A + 1)], ALIGN),
    ([block(m=A + 4)], OVERLAP), ([block(grad=A)], OVERLAP), ([block(weight=A + (2 << 20))], OVERLAP),
    ([block(), block(1, master=A + 16)], OVERLAP), ([block(), block(1, m=A + (2 << 20))], OVERLAP),
])
def test_muon_refuses(rows, code):
    assert muon(rows) == code


def test_muon_refuses_flags_and_workspaces():
    assert muon([block()], edit=lambda a: a.__setitem__("flags", 2)) == INVALID
    assert muon([block()], edit=lambda a: a.__setitem__("reserved", 1)) == INVALID
    assert muon([block()], edit=lambda a: a.__setitem__("weight_dtype", 1)) == DTYPE
    need = lso.muon_workspace_bytes(lso.MuonTable.from_rows([block()]))
    assert muon([block()], nbytes=need - 1) == INVALID
    assert muon([block()], ws=A + (1 << 20) - 256) == OVERLAP
    # gradients may be shared by matrices of one call
    tab = lso.MuonTable.from_rows([block(), block(1, grad=A + (2 << 20))])
    with pytest.raises(lso.LsoError) as e:
        lso.muon_step(tab, WS, 16, stream=0)
    assert "smaller" in str(e.value)


# ----------------------------------------------------------------- embedding

def embed(**kw):
    e = _native.LsoEmbed()
    d = dict(tokens=A, n=10, table=A + (1 << 20), vocab=50, width=24, ld_table=24, rows=A + (2 << 20), ld_rows=24, token_dtype=4,
             table_dtype=2, rows_dtype=2, flags=0, scale=1.0)
    d.update(kw)
    for k, v in d.items():
        setattr(e, k, v)
    return e


BAD_EMBED = [
    (dict(tokens=0), INVALID), (dict(table=0), INVALID), (dict(rows=0), INVALID), (dict(ld_table=23), INVALID),
    (dict(ld_rows=23), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=1e300), INVALID), (dict(n=1 << 31), INVALID),
    (dict(vocab=(1 << 31) - 1), INVALID), (dict(width=1 << 31, ld_table=1 << 31, ld_rows=1 << 31), INVALID), (dict(flags=2), INVALID),
    (dict(token_dtype=1), DTYPE), (dict(table_dtype=0), DTYPE), (dict(rows_dtype=4), DTYPE),
    (dict(tokens=A + 4), ALIGN), (dict(tokens=A + 2, token_dtype=3), ALIGN), (dict(table=A + (1 << 20) + 1), ALIGN),
    (dict(rows=A + (2 << 20) + 2, rows_dtype=1), ALIGN),
    (dict(rows=A + (1 << 20) + 48), OVERLAP), (dict(n=(1 << 31) - 2, width=64, ld_table=64, ld_rows=64, tokens=1 << 44, rows=1 << 46,
                                                    token_dtype=3), INVALID),
]


@pytest.mark.parametrize("kw,code", BAD_EMBED)
def test_embedding_refuses(kw, code):
    lib = _native.lib()
    assert lib.lso_embed_lookup(ctypes.byref(embed(**kw)), None) == code
    assert lib.lso_embed_grad(ctypes.byref(embed(**kw)), WS, 1 << 45, None) == code
    assert lib.lso_last_error()


def test_embedding_refuses_more():
    lib = _native.lib()
    assert lib.lso_embed_lookup(None, None) == INVALID
    assert lib.lso_embed_grad(None, WS, BIG, None) == INVALID
    assert lib.lso_embed_lookup(ctypes.byref(embed(flags=1)), None) == INVALID     # adding is the gradient's
    assert lib.lso_embed_lookup(ctypes.byref(embed(rows=A)), None) == OVERLAP      # the result over the tokens
    assert lib.lso_embed_grad(ctypes.byref(embed(table=A)), WS, BIG, None) == OVERLAP
    need = lso.embed_grad_workspace_bytes(10, 50, 24)
    assert lib.lso_embed_grad(ctypes.byref(embed()), WS, need - 1, None) == INVALID
    assert lib.lso_embed_grad(ctypes.byref(embed()), None, need, None) == INVALID
    assert lib.lso_embed_grad(ctypes.byref(embed()), WS + 4, need, None) == ALIGN
    assert lib.lso_embed_grad(ctypes.byref(embed()), A, need, None) == OVERLAP
    assert lso.embed_grad_workspace_bytes(1 << 31, 1, 1) == 0
    assert lso.embed_grad_workspace_bytes(0, 50, 24) == 0
    # nothing to do
    for kw in (dict(width=0), dict(vocab=0)):
        assert lib.lso_embed_lookup(ctypes.byref(embed(**kw)), None) == 0
        assert lib.lso_embed_grad(ctypes.byref(embed(**kw)), None, 0, None) == 0
    assert lib.lso_embed_lookup(ctypes.byref(embed(n=0)), None) == 0


def test_embedding_producer_refuses():
    lib = _native.lib()
    p = _native.LsoEmbedProducerArgs()
    p.grad, p.embed_layer, p.workspace, p.workspace_bytes = embed(), 3, WS, BIG
    call = lib.lso_embed_producer
    assert call(None, 3, A + (8 << 20), 1200, None) != 0
    assert call(ctypes.addressof(p), 3, A + (8 << 20), 1201, None) != 0    # not vocab * width
    assert call(ctypes.addressof(p), 3, A + (2 << 20), 1200, None) != 0    # over dy
    assert call(ctypes.addressof(p), 2, A + (8 << 20), 1200, None) != 0    # no producer for the other layers
    p.grad.flags = 1
    assert call(ctypes.addressof(p), 3, A + (8 << 20), 1200, None) != 0
    seen = []
    fn = _native.GRAD_FN(lambda u, layer, g, n, s: seen.append((u, layer, g, n, s)) or 7)
    p.other, p.other_user = ctypes.cast(fn, ctypes.c_void_p).value, 99
    assert call(ctypes.addressof(p), 2, A, 5, None) == 7
    assert seen == [(99, 2, A, 5, None)]


def test_embedding_tensor_checks():
    import torch
    w = torch.zeros(5, 8)
    with pytest.raises(ValueError):
        lso.embed_lookup(torch.zeros(3, dtype=torch.int64), w, torch.zeros(3, 8))      # not on a GPU
    with pytest.raises(ValueError):
        ops._embed(torch.zeros(3, dtype=torch.int64), w, torch.zeros(4, 8), 1.0, 0)
    with pytest.raises(ValueError):
        ops._embed(torch.zeros(6, dtype=torch.int64)[::2], w, torch.zeros(3, 8), 1.0, 0)
    with pytest.raises(ValueError):
        ops._embed(torch.zeros(3, dtype=torch.int64), w, torch.zeros(8, 3).T, 1.0, 0)
    with pytest.raises(ValueError):
        ops._embed(torch.zeros(3, dtype=torch.int64), w[0], torch.zeros(3, 8), 1.0, 0)
    with pytest.raises(TypeError):
        lso.dtype_of(torch.zeros(1, dtype=torch.float16))
    assert [lso.dtype_of(torch.zeros(1, dtype=d)) for d in (torch.float32, torch.bfloat16, torch.int32, torch.int64)] == [1, 2, 3, 4]


def test_table_rows():
    tab = lso.MuonTable.from_rows([block(nesterov=False, weight=None), block(1)])
    assert tab.arr["flags"].tolist() == [0, 1] and tab.arr["weight_dtype"].tolist() == [0, 2]
    tab.set_lr(0.5)
    assert np.all(tab.arr["lr"] == 0.5)
    one = lso.MatrixTable.from_rows([mat(), mat(1, ld_x=300)])
    assert one.arr["ld_x"].tolist() == [200, 300] and one.arr["ld_y"].tolist() == [200, 200]


def test_half_precision_is_the_callers_choice():
    """AUTO plans as FULL does, BF16 results or not."""
    for y_dtype in (lso.LSO_DT_F32, lso.LSO_DT_BF16):
        tab = lso.MatrixTable.from_rows([mat(x_dtype=lso.LSO_DT_BF16, y_dtype=y_dtype), mat(1, x_dtype=lso.LSO_DT_BF16, y_dtype=y_dtype)])
        full, half = (lso.orthogonalize_workspace_bytes(tab, p) for p in (lso.LSO_NS_FULL, lso.LSO_NS_HALF))
        assert lso.orthogonalize_workspace_bytes(tab) == full > half


def test_matrix_tables_look_at_tensors():
    """Tensors whose type, shape, strides or place contradict the row are
    refused (CPU tensors here: what is not wrong otherwise fails on that)."""
    import torch
    f, h = torch.zeros(6, 10), torch.zeros(6, 10, dtype=torch.bfloat16)

    def refused(error, match, **kw):
        row = dict(x=f, y=A, rows=6, cols=10)
        row.update(kw)
        with pytest.raises(error, match=match):
            lso.MatrixTable.from_rows([row])
        tab = lso.MatrixTable(1)
        with pytest.raises(error, match=match):
            tab.set_row(0, **row)
        assert tab.arr[0]["rows"] == 0

    refused(TypeError, "y: ", y=h, y_dtype=1)
    refused(TypeError, "x: ", x=f, x_dtype=2)
    refused(TypeError, "float16", x=f.half())
    refused(TypeError, "x: .*int32", x=f.int())
    refused(TypeError, "x: .*int16", x=f.short(), x_dtype=1)
    refused(ValueError, "contiguous", x=torch.zeros(10, 6).T)
    refused(ValueError, "row stride 10 given", x=torch.zeros(6, 12)[:, :10], ld_x=10)
    refused(ValueError, "does not hold", x=f[:5])
    refused(ValueError, "does not hold", x=f, ld_x=11, rows=6, cols=9)
    refused(ValueError, "does not hold", x=torch.zeros(120)[::2])
    for x, kw in ((f, {}), (f.flatten(), {}), (torch.zeros(6, 12)[:, :10], {}), (torch.zeros(72), dict(ld_x=12)), (h, {}),
                  (f.int(), dict(x_dtype=1)), (f.short(), dict(x_dtype=2))):
        refused(ValueError, "not on a GPU", x=x, **kw)
    assert ops._array(h, "x", None, 1, 6, 10) == (h.data_ptr(), 2, 10)
    assert ops._array(torch.zeros(6, 12)[:, :10], "x", None, 2, 6, 10)[1:] == (1, 12)
    assert ops._array(torch.zeros(72), "x", 1, 2, 6, 10, 12)[1:] == (1, 12)
    assert ops._array(A, "x", None, 2, 6, 10) == (A, 2, 10) and ops._array(None, "x", None, 1, 6, 10) == (0, 1, 10)


def test_muon_tables_look_at_tensors():
    import torch
    f = torch.zeros(64, 96)
    for error, match, kw in ((TypeError, "grad: ", dict(grad=f, grad_dtype=2)), (TypeError, "float64", dict(grad=f.double())),
                             (TypeError, "master: ", dict(master=f.bfloat16())), (TypeError, "weight: ", dict(weight=f)),
                             (ValueError, "m must be contiguous", dict(m=torch.zeros(64, 100)[:, :96])),
                             (ValueError, "grad: .*row must be contiguous", dict(grad=torch.zeros(96, 64).T)),
                             (ValueError, "weight: .*does not hold", dict(weight=f[:63].bfloat16())),
                             (ValueError, "offsets", dict(base=A, grad=f)), (ValueError, "grad is on cpu", dict(grad=f))):
        with pytest.raises(error, match=match):
            lso.MuonTable.from_rows([block(**kw)])
    assert lso.MuonTable.from_rows([block()]).arr["grad_dtype"].tolist() == [2]


def test_workspace_tensors_are_looked_at(monkeypatch):
    """A workspace tensor that is not on a GPU, or holds less than is said."""
    import torch
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    tables = lso.MatrixTable.from_rows([mat()]), lso.MuonTable.from_rows([block()])
    for call in (lambda w, n: lso.orthogonalize(tables[0], w, n, stream=0), lambda w, n: lso.muon_step(tables[1], w, n, stream=0)):
        with pytest.raises(ValueError, match="workspace is on cpu"):
            call(ws, 1 << 20)
    with monkeypatch.context() as patch:
        patch.setattr(ops, "_gpu", lambda x, name: None)     # as if it were on the current GPU
        for call in (lambda w, n: lso.orthogonalize(tables[0], w, n, stream=0), lambda w, n: lso.muon_step(tables[1], w, n, stream=0)):
            for w in (ws, ws[::2], torch.zeros(1 << 18, dtype=torch.int16)):
                with pytest.raises(ValueError, match="holds"):
                    call(w, (1 << 20) + 1 if w is ws else 1 << 19 if w.dtype == torch.uint8 else (1 << 19) + 1)
        assert ops._workspace(ws, 1 << 20) == ws.data_ptr()
    assert ops._workspace(WS, BIG) == WS and ops._workspace(None, 0) is None and ops._workspace(0, 0) is None


def test_embedding_producer_looks_at_tensors(monkeypatch):
    """Tensors that are not on a GPU, or not all on one, are refused when the
    producer is made or given a batch, before a stream could run it."""
    import torch
    t, dy, ws = torch.zeros(3, dtype=torch.int64), torch.zeros(3, 8), torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="tokens is on cpu"):
        lso.EmbedProducer(t, dy, 5, 8, WS, BIG)
    places = {id(t): 0, id(dy): 0, id(ws): 0}
    monkeypatch.setattr(ops, "_gpu", lambda x, name: places[id(x)])
    monkeypatch.setattr(torch.cuda, "current_stream", mock.Mock())
    p = lso.EmbedProducer(t, dy, 5, 8, ws, 64)
    assert p._args.workspace == ws.data_ptr() and p._args.grad.tokens == t.data_ptr()
    with pytest.raises(ValueError, match="holds"):
        lso.EmbedProducer(t, dy, 5, 8, ws, 65)
    places[id(ws)] = 1
    with pytest.raises(ValueError, match="workspace is on GPU 1"):
        lso.EmbedProducer(t, dy, 5, 8, ws, 64)
    for x in (t, dy):
        places[id(x)] = 1
        with pytest.raises(ValueError, match="must be on GPU 0"):
            p.set_batch(t, dy)
        places[id(x)] = 0
    p.set_batch(t, dy)
    monkeypatch.undo()
    with pytest.raises(ValueError, match="is on cpu"):
        p.set_batch(t, dy)


def test_embedding_producer_waits_for_its_tensors(monkeypatch):
    """The layer stream's streams wait for no other, so the producer waits for
    the work that writes its batch."""
    import torch
    t, dy, seen = torch.zeros(3, dtype=torch.int64), torch.zeros(3, 8), []

    class Stream:
        def __init__(self, device):
            self.device = device

        def synchronize(self):
            seen.append(self.device)
    monkeypatch.setattr(ops, "_gpu", lambda x, name: 2)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    p = lso.EmbedProducer(t, dy, 5, 8, WS, BIG)
    assert seen == [2]
    p.set_batch(t, dy)
    assert seen == [2, 2]


def test_matrix_tables_refuse_tensors_of_another_shape():
    """A matrix given with its sides exchanged is not read as another one."""
    import torch
    for x, kw in ((torch.zeros(10, 6), {}), (torch.zeros(10, 6), dict(ld_x=10)), (torch.zeros(5, 12), {}), (torch.zeros(1, 60), {}),
                  (torch.zeros(6, 12), dict(ld_x=11))):
        with pytest.raises(ValueError, match="does not hold 6 x 10"):
            lso.MatrixTable.from_rows([dict(x=x, y=A, rows=6, cols=10, **kw)])
    with pytest.raises(ValueError, match="grad: .* does not hold 64 x 96"):
        lso.MuonTable.from_rows([block(grad=torch.zeros(96, 64))])
    for x, kw in ((torch.zeros(6, 12), dict(ld=12)), (torch.zeros(60), {}), (torch.zeros(6, 5, 2), {})):
        assert ops._array(x, "x", None, 2, 6, 10, **kw) == (x.data_ptr(), 1, kw.get("ld", 10))
