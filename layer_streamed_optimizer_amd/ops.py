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


class _Table:
    DTYPE: np.dtype

    def __init__(self, n: int):
        self.arr = np.zeros(n, self.DTYPE)

    def __len__(self) -> int:
        return len(self.arr)

    @classmethod
    def from_rows(cls, rows: Iterable[dict]):
        fields = [cls._fields(**r) for r in rows]
        tab = cls(len(fields))
        tab.arr[:] = fields
        return tab

    @property
    def ptr(self) -> int:
        return self.arr.ctypes.data


class MatrixTable(_Table):
    """A reusable lso_matrix table."""

    DTYPE = MATRIX_DTYPE

    @staticmethod
    def _fields(*, x, y, rows: int, cols: int, ld_x: int | None = None, ld_y: int | None = None, x_dtype: int = LSO_DT_F32,
                y_dtype: int = LSO_DT_F32) -> tuple:
        return (_addr(x), _addr(y), rows, cols, cols if ld_x is None else ld_x, cols if ld_y is None else ld_y, x_dtype, y_dtype)

    def set_row(self, i: int, **row) -> None:
        """x, y (torch tensors, by their data_ptr, or device addresses), rows,
        cols, ld_x, ld_y (default cols), x_dtype, y_dtype (default FP32)."""
        self.arr[i] = self._fields(**row)


class MuonTable(_Table):
    """A reusable lso_muon_block table (lr and the like may be rewritten in
    arr between steps)."""

    DTYPE = MUON_DTYPE

    @staticmethod
    def _fields(*, rows: int, cols: int, master, m, grad, weight=None, base: int = 0, grad_dtype: int = LSO_DT_BF16,
                nesterov: bool = True, lr: float = 1e-3, beta: float = 0.95, weight_decay: float = 0.0, scale: float = 1.0) -> tuple:
        return (base, rows, cols, _addr(master), _addr(m), _addr(grad), _addr(weight), grad_dtype,
                LSO_DT_BF16 if weight is not None else LSO_DT_NONE, LSO_MUON_NESTEROV if nesterov else 0, 0, lr, beta, weight_decay,
                scale)

    def set_row(self, i: int, **row) -> None:
        """rows, cols; master, m, grad and weight (or None): torch tensors or
        device addresses (offsets from base if base != 0); grad_dtype,
        nesterov, lr, beta, weight_decay, scale."""
        self.arr[i] = self._fields(**row)

    def set_lr(self, lr: float) -> None:
        self.arr["lr"] = lr


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
    st = getattr(_native.lib(), name)(table.ptr, len(table), ctypes.byref(p), _addr(workspace) or None, int(workspace_bytes),
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
    """grad[v] = scale * sum of dy[i] over the positions i of token v (+= with
    accumulate), every row of grad written.  Torch tensors; asynchronous."""
    e = _embed(tokens, grad, dy, scale, LSO_EMBED_ADD if accumulate else 0)
    st = _native.lib().lso_embed_grad(ctypes.byref(e), _addr(workspace) or None, int(workspace_bytes), stream_handle(stream))
    if st:
        _native.check(st, "lso_embed_grad")


class EmbedProducer:
    """The gradient producer of a layer stream whose layer `embed_layer` is
    the embedding table of vocab x width parameters:

        p = EmbedProducer(tokens, dy, vocab, width, workspace, nbytes, embed_layer=0, other=fn)
        ls = LayerStream(max_layer_bytes, max_layer_params, p.fn, p.user)

    grad_dtype is the embedding layer's (LSO_DT_BF16 or LSO_DT_F32); other:
    the producer of the other layers (a C function pointer, called with
    other_user).  The tensors and this object must live as long as the
    stream uses them; set_batch takes the next batch's."""

    def __init__(self, tokens, dy, vocab: int, width: int, workspace, workspace_bytes: int, *, embed_layer: int = 0,
                 grad_dtype: int = LSO_DT_BF16, scale: float = 1.0, other: int = 0, other_user: int = 0):
        self._args = LsoEmbedProducerArgs()
        self._shape = (vocab, width)
        self._grad_dtype, self._scale = grad_dtype, scale
        a = self._args
        a.embed_layer = embed_layer
        a.workspace, a.workspace_bytes = _addr(workspace) or None, int(workspace_bytes)
        a.other, a.other_user = other or None, other_user or None
        self.set_batch(tokens, dy)
        self.fn = ctypes.cast(_native.lib().lso_embed_producer, ctypes.c_void_p).value
        self.user = ctypes.addressof(a)

    def set_batch(self, tokens, dy) -> None:
        vocab, width = self._shape
        if not tokens.is_contiguous() or dy.dim() != 2 or tuple(dy.shape) != (tokens.numel(), width):
            raise ValueError("tokens must be contiguous and dy [tokens, width]")
        if dy.shape[0] > 0 and width > 1 and dy.stride(1) != 1:
            raise ValueError("dy: the elements of a row must be contiguous")
        e = self._args.grad
        e.tokens, e.n, e.token_dtype = tokens.data_ptr() or None, tokens.numel(), dtype_of(tokens)
        e.rows, e.rows_dtype = dy.data_ptr() or None, dtype_of(dy)
        e.ld_rows = dy.stride(0) if tokens.numel() > 1 else width
        e.vocab, e.width, e.ld_table, e.table_dtype = vocab, width, width, self._grad_dtype
        e.scale = self._scale
        self._keep = (tokens, dy)
