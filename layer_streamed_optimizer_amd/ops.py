"""The operators of include/lso_ops.h: matrix orthogonalisation, the
orthogonalised-momentum update and the embedding table (marshalling only).

    tab = MuonTable.from_rows([...])              # one dict per weight matrix
    ws = torch.empty(muon_workspace_bytes(tab), dtype=torch.uint8, device="cuda")
    muon_step(tab, ws, ws.numel(), stream)        # momentum, orthogonalisation, write-back

    embed_lookup(tokens, weight, out, scale=s)    # out[i] = s * weight[tokens[i]]
    embed_grad(tokens, dy, grad, ws, ws_bytes, scale=s)
"""
from __future__ import annotations

import ctypes
from typing import Iterable

import numpy as np

from . import _addr, _native, stream_handle
from ._native import (LSO_DT_BF16, LSO_DT_F32, LSO_DT_I32, LSO_DT_I64, LSO_DT_NONE, LSO_EMBED_ADD, LSO_MUON_NESTEROV,
                      LSO_NS_AUTO, LSO_NS_FULL, LSO_NS_HALF, LsoEmbed, LsoEmbedProducerArgs, LsoMatrix, LsoMuonBlock,
                      LsoNsParams)

MATRIX_DTYPE = np.dtype(LsoMatrix)
MUON_DTYPE = np.dtype(LsoMuonBlock)


_codes: dict = {}


def dtype_of(tensor) -> int:
    """The LSO_DT_* code of a torch tensor's dtype."""
    if not _codes:
        import torch
        _codes.update({torch.float32: LSO_DT_F32, torch.bfloat16: LSO_DT_BF16, torch.int32: LSO_DT_I32, torch.int64: LSO_DT_I64})
    code = _codes.get(tensor.dtype)
    if code is None:
        raise TypeError(f"dtype {tensor.dtype} is not one of {', '.join(str(d) for d in _codes)}")
    return code


def _array(x, name: str, code: int | None, default: int, rows: int, cols: int, ld: int | None = None) -> tuple:
    """(address, LSO_DT_* code, row stride) of a matrix's array.  An address
    has the type and stride that are given, or `default` and cols.  A torch
    tensor of shape [rows, cols] brings both; a contiguous one of shape
    [rows, ld], or of one or more than two dimensions, that holds them may
    stand for the rows at stride ld, and one of integers of the same size for
    their bits.  What contradicts the tensor is refused."""
    if x is None or isinstance(x, int):
        return x or 0, default if code is None else code, cols if ld is None else ld
    addr, dtype = x.data_ptr(), x.dtype
    if code is None or dtype.is_floating_point:
        own = dtype_of(x)
        if own != LSO_DT_F32 and own != LSO_DT_BF16 or code is not None and code != own:
            raise TypeError(f"{name}: a tensor of {dtype}" + ("" if code is None else f" given as type code {code}"))
    else:
        own = code
        if x.element_size() != (4 if code == LSO_DT_F32 else 2):
            raise TypeError(f"{name}: a tensor of {x.dtype} cannot hold the bits of type code {code}")
    if rows == 0 or cols == 0:
        return addr, own, cols if ld is None else ld
    if x.shape == (rows, cols):
        in_rows, in_cols = x.stride()
        if cols > 1 and in_cols != 1:
            raise ValueError(f"{name}: the elements of a row must be contiguous (strides {in_rows}, {in_cols})")
        if rows > 1:
            if ld is not None and ld != in_rows:
                raise ValueError(f"{name}: row stride {ld} given for a tensor of row stride {in_rows}")
            ld = in_rows
    elif (not x.is_contiguous() or x.numel() < (rows - 1) * (cols if ld is None else ld) + cols
          or x.dim() == 2 and x.shape != (rows, ld)):
        raise ValueError(f"{name}: a tensor of shape {tuple(x.shape)} and strides {x.stride()} does not hold {rows} x {cols}")
    return addr, own, cols if ld is None else ld


def _gpu(x, name: str) -> int | None:
    """The GPU of a torch tensor; None for an address."""
    if x is None or isinstance(x, int):
        return None
    if not x.is_cuda:
        raise ValueError(f"{name} is on {x.device}, not on a GPU")
    return x.get_device()


def _check_device(device: int | None) -> None:
    """device: of a call's tensors, or None."""
    if device is None:
        return
    global _current_device
    if _current_device is None:
        import torch
        _current_device = torch.cuda.current_device
    if device != _current_device():
        raise ValueError(f"the tensors are on GPU {device}, which is not the current device")


_current_device = None


class _Table:
    """Rows hold addresses: the tensors that they were made from must live as
    long as the table is used."""

    DTYPE: np.dtype

    def __init__(self, n: int):
        self.arr = np.zeros(n, self.DTYPE)
        self.device: int | None = None     # of the tensors that its rows were made from

    def __len__(self) -> int:
        return len(self.arr)

    @classmethod
    def from_rows(cls, rows: Iterable[dict]):
        rows = list(rows)
        tab = cls(len(rows))
        tab.arr[:] = [tab._row(**r) for r in rows]
        return tab

    def _row(self, **row) -> tuple:
        fields, arrays = self._fields(**row)
        for name, x in arrays:
            device = _gpu(x, name)
            if device is None:
                continue
            if self.device is None:
                self.device = device
            elif device != self.device:
                raise ValueError(f"{name} is on GPU {device}, the table's other tensors on GPU {self.device}")
        return fields

    @property
    def ptr(self) -> int:
        return self.arr.ctypes.data


class MatrixTable(_Table):
    """A reusable lso_matrix table."""

    DTYPE = MATRIX_DTYPE

    @staticmethod
    def _fields(*, x, y, rows: int, cols: int, ld_x: int | None = None, ld_y: int | None = None, x_dtype: int | None = None,
                y_dtype: int | None = None) -> tuple:
        ax, tx, lx = _array(x, "x", x_dtype, LSO_DT_F32, rows, cols, ld_x)
        ay, ty, ly = _array(y, "y", y_dtype, LSO_DT_F32, rows, cols, ld_y)
        return (ax, ay, rows, cols, lx, ly, tx, ty), (("x", x), ("y", y))

    def set_row(self, i: int, **row) -> None:
        """x, y, rows, cols, ld_x, ld_y, x_dtype, y_dtype.  x and y are torch
        tensors, which bring their type and row stride, or device addresses
        (FP32 and cols unless given)."""
        self.arr[i] = self._row(**row)


class MuonTable(_Table):
    """A reusable lso_muon_block table (lr and the like may be rewritten in
    arr between steps)."""

    DTYPE = MUON_DTYPE

    @staticmethod
    def _fields(*, rows: int, cols: int, master, m, grad, weight=None, base: int = 0, grad_dtype: int | None = None,
                nesterov: bool = True, lr: float = 1e-3, beta: float = 0.95, weight_decay: float = 0.0, scale: float = 1.0) -> tuple:
        arrays = (("master", master), ("m", m), ("grad", grad), ("weight", weight))
        addr = []
        for (name, a), code, default in zip(arrays, (LSO_DT_F32, LSO_DT_F32, grad_dtype, LSO_DT_BF16),
                                            (LSO_DT_F32, LSO_DT_F32, LSO_DT_BF16, LSO_DT_BF16)):
            at, own, ld = _array(a, name, code, default, rows, cols)
            if ld != cols and rows > 1:
                raise ValueError(f"{name} must be contiguous (row stride {ld})")
            if base != 0 and a is not None and not isinstance(a, int):
                raise ValueError(f"{name}: with a base, arrays are offsets from it, not tensors")
            addr.append(at)
            if name == "grad":
                grad_dtype = own
        return (base, rows, cols, *addr, grad_dtype, LSO_DT_BF16 if weight is not None else LSO_DT_NONE,
                LSO_MUON_NESTEROV if nesterov else 0, 0, lr, beta, weight_decay, scale), arrays

    def set_row(self, i: int, **row) -> None:
        """rows, cols; master, m, grad and weight (or None): contiguous torch
        tensors or device addresses (offsets from base if base != 0);
        grad_dtype (the tensor's, or BF16 for an address), nesterov, lr, beta,
        weight_decay, scale."""
        self.arr[i] = self._row(**row)

    def set_lr(self, lr: float) -> None:
        self.arr["lr"] = lr


def _workspace(workspace, nbytes: int, device: int | None = None) -> int | None:
    """The address of a workspace; a torch tensor has to hold nbytes on the
    current device (or on the one given)."""
    if workspace is None or isinstance(workspace, int):
        return workspace or None
    at = _gpu(workspace, "the workspace")
    if device is None:
        _check_device(at)
    elif at != device:
        raise ValueError(f"the workspace is on GPU {at}, the tokens on GPU {device}")
    if not workspace.is_contiguous() or workspace.nbytes < nbytes:
        raise ValueError(f"the workspace tensor holds {workspace.nbytes} contiguous bytes, not the {nbytes} given")
    return workspace.data_ptr() or None


def _params(steps: int, eps: float, coefficients, precision: int):
    """lso_ns_params and the array it points into (to be kept alive)."""
    coef = None
    if coefficients is not None:
        coef = np.ascontiguousarray(coefficients, dtype=np.float64)
        if coef.shape == (3,):
            coef = np.tile(coef, (max(steps, 1), 1))
        if coef.shape != (steps, 3):
            raise ValueError("coefficients: one triple, or one for each step")
    if not 0 <= steps < 1 << 32:
        raise ValueError("steps out of range")
    return LsoNsParams(steps, precision, eps, coef.ctypes.data if coef is not None else None), coef


def _run(name: str, table: _Table, workspace, workspace_bytes: int, steps, eps, coefficients, precision, stream) -> None:
    p, keep = _params(steps, eps, coefficients, precision)
    _check_device(table.device)
    st = getattr(_native.lib(), name)(table.ptr, len(table), ctypes.byref(p), _workspace(workspace, workspace_bytes), int(workspace_bytes),
                                      stream_handle(stream))
    if st:
        _native.check(st, name)


def _bytes(name: str, table: _Table, precision: int) -> int:
    p = LsoNsParams(5, precision, 1e-7, None)
    need = int(getattr(_native.lib(), name)(table.ptr, len(table), ctypes.byref(p)))
    if need == 0 and _native.lib().lso_last_error():
        _native.check(_native.LSO_E_INVALID, name)
    return need


def orthogonalize_workspace_bytes(table: MatrixTable, precision: int = LSO_NS_AUTO) -> int:
    """Device workspace orthogonalize needs for this table."""
    return _bytes("lso_orthogonalize_workspace_bytes", table, precision)


def orthogonalize(table: MatrixTable, workspace, workspace_bytes: int, *, steps: int = 5, eps: float = 1e-7,
                  coefficients=None, precision: int = LSO_NS_AUTO, stream=None) -> None:
    """y of every matrix of the table from its x by `steps` Newton-Schulz
    steps.  coefficients: (a, b, c), or one such triple for each step.
    Asynchronous."""
    _run("lso_orthogonalize", table, workspace, workspace_bytes, steps, eps, coefficients, precision, stream)


def muon_workspace_bytes(table: MuonTable, precision: int = LSO_NS_AUTO) -> int:
    """Device workspace muon_step needs for this table."""
    return _bytes("lso_muon_workspace_bytes", table, precision)


def muon_step(table: MuonTable, workspace, workspace_bytes: int, *, steps: int = 5, eps: float = 1e-7, coefficients=None,
              precision: int = LSO_NS_AUTO, stream=None) -> None:
    """One orthogonalised-momentum update of every matrix of the table.
    Asynchronous."""
    _run("lso_muon_step", table, workspace, workspace_bytes, steps, eps, coefficients, precision, stream)


# ------------------------------------------------------------------ embedding

def _embed(tokens, table, rows, scale: float, flags: int) -> LsoEmbed:
    """The descriptor of torch tensors: tokens (any shape, contiguous), table
    [vocab, width], rows [..., width] with one position after another."""
    if table.dim() != 2:
        raise ValueError("the table must have two dimensions")
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    n, (vocab, width) = tokens.numel(), table.shape
    if rows.dim() < 1 or rows.shape[-1] != width or rows.numel() != n * width:
        raise ValueError(f"rows of shape {tuple(rows.shape)} do not match {n} tokens of width {width}")
    if rows.dim() != 2:
        rows = rows.view(n, width)   # raises if the positions are not evenly spaced
    ld_table, in_table = table.stride()
    ld_rows, in_rows = rows.stride()
    if width > 1 and ((vocab > 0 and in_table != 1) or (n > 0 and in_rows != 1)):
        raise ValueError("the elements of a row must be contiguous")
    device = tokens.device
    if device.type != "cuda" or table.device != device or rows.device != device:
        raise ValueError("tokens, table and rows must be on one GPU")
    import torch
    if device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {device}, which is not the current device")
    return LsoEmbed(tokens.data_ptr(), n, table.data_ptr(), vocab, width, ld_table if vocab > 1 else width, rows.data_ptr(),
                    ld_rows if n > 1 else width, dtype_of(tokens), dtype_of(table), dtype_of(rows), flags, scale)


_lookup_fn = None


def embed_lookup(tokens, weight, out, *, scale: float = 1.0, stream=None) -> None:
    """out[i] = scale * weight[tokens[i]] (a zero row where the token is
    outside the table).  Torch tensors; asynchronous."""
    global _lookup_fn
    if _lookup_fn is None:
        _lookup_fn = _native.lib().lso_embed_lookup
    e = _embed(tokens, weight, out, scale, 0)
    st = _lookup_fn(ctypes.byref(e), stream_handle(stream))
    if st:
        _native.check(st, "lso_embed_lookup")


def embed_grad_workspace_bytes(n_tokens: int, vocab: int, width: int) -> int:
    """Device workspace embed_grad needs."""
    return int(_native.lib().lso_embed_grad_workspace_bytes(n_tokens, vocab, width))


def embed_grad(tokens, dy, grad, workspace, workspace_bytes: int, *, scale: float = 1.0, accumulate: bool = False,
               stream=None) -> None:
    """grad[v] = scale * sum of dy[i] over the positions i of token v; every row
    of grad is written, zeros where a token does not occur.  With accumulate,
    += that, and such rows are left as they are.  Torch tensors;
    asynchronous."""
    e = _embed(tokens, grad, dy, scale, LSO_EMBED_ADD if accumulate else 0)
    st = _native.lib().lso_embed_grad(ctypes.byref(e), _workspace(workspace, workspace_bytes), int(workspace_bytes), stream_handle(stream))
    if st:
        _native.check(st, "lso_embed_grad")


class EmbedProducer:
    """The gradient producer of a layer stream whose layer `embed_layer` is
    the embedding table of vocab x width parameters:

        p = EmbedProducer(tokens, dy, vocab, width, workspace, nbytes, embed_layer=0, other=fn)
        ls = LayerStream(max_layer_bytes, max_layer_params, p.fn, p.user)

    grad_dtype is the embedding layer's (LSO_DT_BF16 or LSO_DT_F32); other:
    the producer of the other layers (a C function pointer, called with
    other_user).  The tensors are on the stream's GPU; they and this object
    must live as long as the stream uses them.  A layer stream's own streams
    wait for no other: set_batch, which takes the next batch's tensors,
    returns when the work of torch's current stream so far is done, and
    whoever refills the same tensors calls it again."""

    def __init__(self, tokens, dy, vocab: int, width: int, workspace, workspace_bytes: int, *, embed_layer: int = 0,
                 grad_dtype: int = LSO_DT_BF16, scale: float = 1.0, other: int = 0, other_user: int = 0):
        self._args = LsoEmbedProducerArgs()
        self._shape = (vocab, width)
        self._grad_dtype, self._scale = grad_dtype, scale
        a = self._args
        a.embed_layer = embed_layer
        a.other, a.other_user = other or None, other_user or None
        self._device = _gpu(tokens, "tokens")
        self.set_batch(tokens, dy)
        a.workspace, a.workspace_bytes = _workspace(workspace, workspace_bytes, self._device), int(workspace_bytes)
        self._workspace = workspace
        self.fn = ctypes.cast(_native.lib().lso_embed_producer, ctypes.c_void_p).value
        self.user = ctypes.addressof(a)

    def set_batch(self, tokens, dy) -> None:
        vocab, width = self._shape
        if not tokens.is_contiguous() or dy.dim() != 2 or tuple(dy.shape) != (tokens.numel(), width):
            raise ValueError("tokens must be contiguous and dy [tokens, width]")
        if dy.shape[0] > 0 and width > 1 and dy.stride(1) != 1:
            raise ValueError("dy: the elements of a row must be contiguous")
        if _gpu(tokens, "tokens") != self._device or _gpu(dy, "dy") != self._device:
            raise ValueError(f"tokens and dy must be on GPU {self._device}, where the first batch was")
        e = self._args.grad
        e.tokens, e.n, e.token_dtype = tokens.data_ptr() or None, tokens.numel(), dtype_of(tokens)
        e.rows, e.rows_dtype = dy.data_ptr() or None, dtype_of(dy)
        e.ld_rows = dy.stride(0) if tokens.numel() > 1 else width
        e.vocab, e.width, e.ld_table, e.table_dtype = vocab, width, width, self._grad_dtype
        e.scale = self._scale
        self._keep = (tokens, dy)
        if self._device is not None:
            import torch
            torch.cuda.current_stream(self._device).synchronize()
