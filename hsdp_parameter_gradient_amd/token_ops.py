"""The token operators: embedding lookup and norm, with their gradients.

What a layer does between the full parameters of a bucket (AG copy-out) and
its full gradients (RS copy-in, or the fused RS copy-reduce), apart from the
matrix products: thin wrappers of the C entry points of the same names, which
check and marshal their tensors as _binding does.  Activations are dense
tensors [..., cols]; the simulated ranks' rows stand one rank after the other,
and a gradient call writes one parameter gradient per rank.

A gradient call needs a workspace.  It is allocated through torch on the
stream of the call and given back when the call has been issued; a prepared
call (prepare) keeps its own, so it must not overlap in time with itself.
"""

from __future__ import annotations

import ctypes
from ctypes import c_int64, c_void_p
from typing import Optional, Sequence

import torch

from . import _binding as B

LAYER = "layer"
RMS = "rms"
_KINDS = {LAYER: 0, RMS: 1}


class Dropout:
    """Dropout with a mask that is drawn from (seed, step, site) and the
    element's place, and never stored.

    p: the probability of dropping, in [0, 1), used as a multiple of 2^-16;
    state: int64 device tensor [2], seed and step, read by the kernels (add 1
    to state[1] after every training step, in a captured one too);
    site: tells the dropouts of one step apart.  The gradient of a call takes
    the Dropout that the call took, with the same seed and step."""

    __slots__ = ("p", "state", "site", "struct", "ref")

    def __init__(self, p: float, state: torch.Tensor, site: int = 0):
        if not 0.0 <= p < 1.0 or int(p * 65536 + 0.5) == 65536:
            raise ValueError(f"dropout p {p}: expected [0, 1) (a multiple of 2^-16)")
        if not 0 <= site < 1 << 32:
            raise ValueError(f"dropout site {site}: expected 32 bits")
        self.p, self.state, self.site = p, state, site
        self.struct = B._Dropout(p, site, B._dev(state, "dropout state", 2, torch.int64))
        self.ref = ctypes.byref(self.struct)


def _tokens(tokens: torch.Tensor) -> int:
    """The bytes of one token."""
    if not isinstance(tokens, torch.Tensor) or tokens.dtype not in (torch.int64, torch.int32):
        raise ValueError("tokens: expected an int64 or int32 device tensor")
    return tokens.dtype.itemsize


def _opt(t: Optional[torch.Tensor], what: str, numel: int, dtype: torch.dtype) -> Optional[int]:
    return None if t is None else B._dev(t, what, numel, dtype) or None


def _grads(grads: Sequence[torch.Tensor], what: str, n_ranks: int, numel: int, dtype: torch.dtype):
    if len(grads) != n_ranks:
        raise ValueError(f"{what}: {len(grads)} tensors, expected {n_ranks}")
    return B._ptr_array([B._dev(t, f"{what}[{g}]", numel, dtype) for g, t in enumerate(grads)])


def _prep_embedding(tokens, table, out, scale=1.0, dropout=None):
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table: expected a [vocab, cols] tensor")
    V, E = table.shape
    nb, T = _tokens(tokens), tokens.numel()
    args = (V, E, B._dtype_code(table.dtype), B._dtype_code(out.dtype), B._dev(table, "table", V * E) or None, T, nb,
            B._dev(tokens, "tokens", T) or None, scale, dropout.ref if dropout is not None else None,
            B._dev(out, "out", T * E) or None)
    return B._Call("fsdp_embedding", args, (tokens, table, out, dropout.state if dropout is not None else None, dropout))


class _WorkspaceCall(B._Call):
    """A marshalled call whose workspace is still to be allocated: at[0] is
    the workspace's place among the arguments, nbytes its size."""

    def __init__(self, name, args, keep, at, nbytes):
        super().__init__(name, args, keep)
        self.at, self.nbytes, self.workspace = at, nbytes, None

    def allocate(self, stream=None):
        """Allocate the workspace for a launch on `stream` (default: the
        current one), from that stream's share of torch's memory."""
        if stream is None:
            ws = torch.empty(self.nbytes, dtype=torch.uint8, device=torch.device("cuda", self.device))
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=torch.device("cuda", self.device)) if int(stream) else \
                    torch.cuda.default_stream(self.device)
            with torch.cuda.stream(stream):
                ws = torch.empty(self.nbytes, dtype=torch.uint8, device=torch.device("cuda", self.device))
        self.workspace = ws
        a = list(self.args)
        a[self.at] = ws.data_ptr()
        self.args = tuple(a)

    def keep_workspace(self):
        """For prepared calls: a workspace that lives as long as the call and
        serves whatever stream the call is issued on (what used its memory
        before has ended)."""
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError(f"{self.name}: prepare the call before the capture (its workspace outlives the graph)")
        self.workspace = torch.empty(self.nbytes, dtype=torch.uint8, device=torch.device("cuda", self.device))
        torch.cuda.current_stream(self.device).synchronize()
        a = list(self.args)
        a[self.at] = self.workspace.data_ptr()
        self.args = tuple(a)
        return self

    def once(self, stream):
        self.allocate(stream)
        self(stream)


def fsdp_embedding_grad_workspace(n_ranks: int, n_tokens: int, vocab: int, cols: int) -> int:
    """Bytes of fsdp_embedding_grad's workspace (n_tokens of one rank)."""
    n = c_int64()
    B._check("fsdp_embedding_grad_workspace",
             B.lib().fsdp_embedding_grad_workspace(n_ranks, n_tokens, vocab, cols, ctypes.byref(n)))
    return n.value


def fsdp_norm_grad_workspace(n_ranks: int, rows: int, cols: int) -> int:
    """Bytes of fsdp_norm_grad's workspace (rows of one rank)."""
    n = c_int64()
    B._check("fsdp_norm_grad_workspace", B.lib().fsdp_norm_grad_workspace(n_ranks, rows, cols, ctypes.byref(n)))
    return n.value


def _marshal_embedding_grad(tokens, dout, grads, scale=1.0, dropout=None, accumulate=False):
    R = len(grads)
    if R < 1:
        raise ValueError("grads: expected one tensor per rank")
    nb, n = _tokens(tokens), tokens.numel()
    if n % R:
        raise ValueError(f"tokens: {n} elements for {R} ranks")
    if not isinstance(dout, torch.Tensor) or dout.dim() < 1:
        raise ValueError("dout: expected a [..., cols] tensor")
    E = dout.shape[-1]
    if E < 1 or grads[0].numel() % E:
        raise ValueError(f"grads[0]: {grads[0].numel()} elements are no rows of {E}")
    V, T, gd = grads[0].numel() // E, n // R, grads[0].dtype
    arr = _grads(grads, "grads", R, V * E, gd)
    nbytes = fsdp_embedding_grad_workspace(R, T, V, E)
    args = (R, V, E, B._dtype_code(dout.dtype), B._dtype_code(gd), T, nb, B._dev(tokens, "tokens", n) or None,
            B._dev(dout, "dout", n * E) or None, scale, dropout.ref if dropout is not None else None,
            int(bool(accumulate)), arr, None, nbytes)
    keep = (tokens, dout, tuple(grads), dropout.state if dropout is not None else None, dropout, arr)
    return _WorkspaceCall("fsdp_embedding_grad", args, keep, 13, nbytes)


def _kind(kind: str) -> int:
    if kind not in _KINDS:
        raise ValueError(f"norm kind {kind!r}: expected {LAYER!r} or {RMS!r}")
    return _KINDS[kind]


def _rows(x: torch.Tensor, weight: torch.Tensor, what: str):
    if not isinstance(x, torch.Tensor) or not isinstance(weight, torch.Tensor):
        raise TypeError(f"{what}, weight: expected torch.Tensors")
    E = weight.numel()
    if E < 1 or x.dim() < 1 or x.shape[-1] != E:
        raise ValueError(f"{what}: last dim of {tuple(x.shape)} is not the weight's {E}")
    return x.numel() // E, E


def _prep_norm(x, weight, y, bias=None, residual=None, h=None, mean=None, rstd=None, eps=1e-5, kind=LAYER,
               dropout=None):
    k, (n, E), dt, f32 = _kind(kind), _rows(x, weight, "x"), x.dtype, torch.float32
    args = (k, n, E, B._dtype_code(dt), B._dtype_code(weight.dtype), B._dev(x, "x", n * E) or None,
            _opt(residual, "residual", n * E, dt), dropout.ref if dropout is not None else None,
            B._dev(weight, "weight", E), _opt(bias, "bias", E, weight.dtype), eps, _opt(h, "h", n * E, dt),
            B._dev(y, "y", n * E, dt) or None, _opt(mean, "mean", n, f32), _opt(rstd, "rstd", n, f32))
    return B._Call("fsdp_norm", args, (x, weight, y, bias, residual, h, mean, rstd,
                                       dropout.state if dropout is not None else None, dropout))


def _marshal_norm_grad(dy, h, rstd, weight, dres, dweight, mean=None, dbias=None, dh=None, dx=None, kind=LAYER,
                       dropout=None, accumulate=False):
    k, (n, E), dt, f32 = _kind(kind), _rows(dy, weight, "dy"), dy.dtype, torch.float32
    R = len(dweight)
    if R < 1 or n % R:
        raise ValueError(f"dweight: {R} tensors for {n} rows: expected one per rank")
    if mean is None and k == 0:
        raise ValueError("mean: the layer norm's gradient needs it")
    T, gd = n // R, dweight[0].dtype
    warr = _grads(dweight, "dweight", R, E, gd)
    barr = _grads(dbias, "dbias", R, E, gd) if dbias is not None else None
    nbytes = fsdp_norm_grad_workspace(R, T, E)
    args = (k, R, T, E, B._dtype_code(dt), B._dtype_code(weight.dtype), B._dtype_code(gd),
            B._dev(dy, "dy", n * E) or None, _opt(dh, "dh", n * E, dt), B._dev(h, "h", n * E, dt) or None,
            _opt(mean, "mean", n, f32), B._dev(rstd, "rstd", n, f32) or None, B._dev(weight, "weight", E),
            dropout.ref if dropout is not None else None, int(bool(accumulate)),
            B._dev(dres, "dres", n * E, dt) or None, _opt(dx, "dx", n * E, dt), warr, barr, None, nbytes)
    keep = (dy, h, rstd, weight, dres, tuple(dweight), mean, tuple(dbias or ()), dh, dx,
            dropout.state if dropout is not None else None, dropout, warr, barr)
    return _WorkspaceCall("fsdp_norm_grad", args, keep, 19, nbytes)


B._PREP.update({
    "fsdp_embedding": _prep_embedding,
    "fsdp_embedding_grad": lambda *a, **k: _marshal_embedding_grad(*a, **k).keep_workspace(),
    "fsdp_norm": _prep_norm,
    "fsdp_norm_grad": lambda *a, **k: _marshal_norm_grad(*a, **k).keep_workspace(),
})


def fsdp_embedding(tokens: torch.Tensor, table: torch.Tensor, out: torch.Tensor, scale: float = 1.0,
                   dropout: Optional[Dropout] = None, stream=None) -> None:
    """out[t] = drop(scale * table[tokens[t]]); a token outside [0, vocab)
    gives a row of zeros.  table: [vocab, cols]; tokens: int64 or int32, any
    shape; out: [..., cols], its dtype may differ from the table's."""
    _prep_embedding(tokens, table, out, scale, dropout)(stream)


def fsdp_embedding_grad(tokens: torch.Tensor, dout: torch.Tensor, grads: Sequence[torch.Tensor], scale: float = 1.0,
                        dropout: Optional[Dropout] = None, accumulate: bool = False, stream=None) -> None:
    """grads[g][v] = scale * the sum of drop'(dout) over rank g's positions
    with token v (added to grads[g][v] if accumulate).  tokens: the R ranks'
    tokens, R = len(grads), one rank after the other; dout: their rows."""
    _marshal_embedding_grad(tokens, dout, grads, scale, dropout, accumulate).once(stream)


def fsdp_norm(x: torch.Tensor, weight: torch.Tensor, y: torch.Tensor, bias: Optional[torch.Tensor] = None,
              residual: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
              mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None, eps: float = 1e-5,
              kind: str = LAYER, dropout: Optional[Dropout] = None, stream=None) -> None:
    """h = residual + drop(x); y = (h - mean) * rstd * weight + bias over the
    last dim (kind RMS: h * rstd * weight, rstd = 1 / rms(h)).  h may be left
    out without a residual and a dropout; mean and rstd (float32, one per row)
    are what the gradient reads."""
    _prep_norm(x, weight, y, bias, residual, h, mean, rstd, eps, kind, dropout)(stream)


def fsdp_norm_grad(dy: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor, dres: torch.Tensor,
                   dweight: Sequence[torch.Tensor], mean: Optional[torch.Tensor] = None,
                   dbias: Optional[Sequence[torch.Tensor]] = None, dh: Optional[torch.Tensor] = None,
                   dx: Optional[torch.Tensor] = None, kind: str = LAYER, dropout: Optional[Dropout] = None,
                   accumulate: bool = False, stream=None) -> None:
    """The norm's gradient: dres that of h (and the residual), dh added to it;
    dx that of x (drop'(dres)); dweight[g] and dbias[g] those of rank g's
    rows, R = len(dweight) ranks one after the other."""
    _marshal_norm_grad(dy, h, rstd, weight, dres, dweight, mean, dbias, dh, dx, kind, dropout, accumulate).once(stream)
