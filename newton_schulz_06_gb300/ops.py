"""Python face of libmuon's operators of a block's training step.

Layer norm, activation checkpoints in 8 bits, the weight gradient read from a
checkpoint, and the router of a mixture-of-experts block with its balance
loss: what leads from a block's activations to the gradients that
:class:`~newton_schulz_06_gb300.muon.Muon` steps with.

    y, rstd, saved = layer_norm_checkpoint(x, weight, bias)   # h kept in 8 bits
    q = y @ Wq.t()
    ...
    weight_grad(dq, saved, weight=weight, bias=bias, out=Gq)  # G that opt.step() reads
    dx, dweight, dbias = layer_norm_backward(dy, saved, None, rstd, weight, bias)

PyTorch supplies device memory and the stream; every value is computed in
libmuon's kernels.  All calls queue their work on the current stream of their
tensors' device and return; outputs that are not given are allocated.
Tensors are CUDA tensors, row-major (stride(1) == 1), fp32 or bf16 as stated;
include/muon.h has each operator's formula.

Nothing here records for torch.autograd: an input's requires_grad has no
effect, and the passes are joined by hand, as examples/train_moe_block.py does.
The bits of a row of the layer norm may depend on the number of rows beside it
and on its alignment (other kernels add in another order); the same call gives
the same bits again.
"""
from __future__ import annotations

import ctypes
import threading
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import MuonError, lib
from .muon import _DT

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
_NO_CKPT = (0, 0, 0, 0)
_ERR_LEN = 256
_norm_args = _lib.packer(_lib.LayerNormArgs).pack
_norm_grad_args = _lib.packer(_lib.LayerNormGradArgs).pack
_weight_grad_args = _lib.packer(_lib.WeightGradArgs).pack
_route_args = _lib.packer(_lib.RouteArgs).pack
_route_grad_args = _lib.packer(_lib.RouteGradArgs).pack
_ckpt_arg = _lib.packer(_lib.Ckpt8).pack


class _Local(threading.local):
    """A thread's message buffer and workspace size."""

    def __init__(self):
        self.err = ctypes.create_string_buffer(_ERR_LEN)
        self.size = ctypes.c_size_t()
        self.size_ref = ctypes.byref(self.size)


_local = _Local()


_fns = {}


def _fn(name: str):
    """An entry point of the library (looked up once)."""
    f = _fns.get(name)
    if f is None:
        f = _fns[name] = getattr(lib(), name)
    return f


def _need(ok: bool, message: str) -> None:
    if not ok:
        raise ValueError(message)


def _dtype(name: str, t: torch.Tensor) -> int:
    d = _DT.get(t.dtype)
    if d is None:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return d


def _matrix(name: str, t: torch.Tensor, index: int = -1, rows: int = -1, cols: int = -1):
    """Checks a row-major 2-D CUDA tensor (of device `index` and rows x cols,
    where given): (rows, cols, leading dimension, device index)."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(shape)}")
    on = t.get_device()
    if on < 0 or (index >= 0 and on != index):
        raise ValueError(f"{name} must be a CUDA tensor of its operator's device, is on {t.device}")
    r, c = shape
    if rows >= 0 and (r != rows or c != cols):
        raise ValueError(f"{name} must be {(rows, cols)}, got {tuple(shape)}")
    ld, inner = t.stride()
    if inner != 1 and c > 1:
        raise ValueError(f"{name} must be row-major (stride(1) == 1)")
    return r, c, ld, on


def _vector(name: str, t: Optional[torch.Tensor], index: int, n: int, dtype=None) -> int:
    """Checks a dense 1-D tensor of n values (or None); its address."""
    if t is None:
        return 0
    if t.dim() != 1 or t.numel() != n or t.get_device() != index or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be {n} dense values on cuda:{index}, got {tuple(t.shape)} "
                         f"on {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _call(index: int, name: str, *args) -> None:
    """Calls an entry point on the device's current stream, with the device
    current."""
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return _call(index, name, *args)
    err = _local.err
    rc = _fn(name)(*args, torch._C._cuda_getCurrentRawStream(index), err, _ERR_LEN)
    if rc < 0:
        raise MuonError(rc, f"{name}: {err.value.decode(errors='replace')}")


def _call_ws(index: int, name: str, query: str, args: bytes, device) -> None:
    """Calls an entry point that takes a workspace, allocated here."""
    size = _local.size
    size.value = 0
    # a query that refuses its arguments leaves the message to the call
    _fn(query)(args, _local.size_ref)
    n = size.value
    if n:
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        _call(index, name, args, ws.data_ptr(), n)
    else:
        _call(index, name, args, None, 0)


class Checkpoint8:
    """An activation checkpoint: rows x cols values in 8 bits, in blocks of 32
    consecutive values of a row that share a power of two (include/muon.h,
    muon_ckpt8).  q: int8, rows x (cols rounded up to 32 or more), e: uint8,
    rows x ceil(cols / 32)."""

    __slots__ = ("q", "e", "cols")

    def __init__(self, q: torch.Tensor, e: torch.Tensor, cols: int):
        blocks = -(-cols // 32)
        if q.dtype != torch.int8 or e.dtype != torch.uint8:
            raise ValueError("q must be int8 and e uint8")
        if q.dim() != 2 or e.dim() != 2 or cols < 1 or q.shape[1] < 32 * blocks \
                or e.shape[1] < blocks or q.shape[0] != e.shape[0]:
            raise ValueError(f"q {tuple(q.shape)} and e {tuple(e.shape)} do not hold {cols} columns")
        if q.stride(1) != 1 or (e.stride(1) != 1 and e.shape[1] > 1) or q.device != e.device:
            raise ValueError("q and e must be row-major and on one device")
        self.q, self.e, self.cols = q, e, cols

    @classmethod
    def empty(cls, rows: int, cols: int, device) -> "Checkpoint8":
        blocks = -(-cols // 32)
        c = cls.__new__(cls)
        c.q = torch.empty((rows, 32 * blocks), dtype=torch.int8, device=device)
        c.e = torch.empty((rows, blocks), dtype=torch.uint8, device=device)
        c.cols = cols
        return c

    @property
    def rows(self) -> int:
        return self.q.shape[0]

    @property
    def shape(self) -> Tuple[int, int]:
        return self.q.shape[0], self.cols

    @property
    def device(self) -> torch.device:
        return self.q.device

    @property
    def nbytes(self) -> int:
        return self.q.nbytes + self.e.nbytes

    def _fields(self):
        return self.q.data_ptr(), self.e.data_ptr(), self.q.stride(0), self.e.stride(0)

    def values(self, dtype: torch.dtype = torch.bfloat16,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """What the checkpoint stands for (exact in bf16 and fp32)."""
        q, cols = self.q, self.cols
        rows = q.shape[0]
        if out is None:
            out = torch.empty((rows, cols), dtype=dtype, device=q.device)
        _, _, ld, index = _matrix("out", out, q.get_device(), rows, cols)
        _call(index, "muon_ckpt8_unpack", _ckpt_arg(*self._fields()), rows, cols, out.data_ptr(),
              _dtype("out", out), ld)
        return out


def checkpoint8(x: torch.Tensor, out: Optional[Checkpoint8] = None) -> Checkpoint8:
    """The 8-bit checkpoint of x (2-D, fp32 or bf16)."""
    rows, cols, ld, index = _matrix("x", x)
    out = _checkpoint("out", out, rows, cols, x)
    _call(index, "muon_ckpt8_pack", x.data_ptr(), _dtype("x", x), rows, cols, ld,
          _ckpt_arg(*out._fields()))
    return out


def _checkpoint(name: str, c: Optional[Checkpoint8], rows: int, cols: int, like) -> Checkpoint8:
    if c is None:
        return Checkpoint8.empty(rows, cols, like.device)
    _need(c.shape == (rows, cols) and c.device == like.device,
          f"{name} must be a checkpoint of {(rows, cols)} on {like.device}")
    return c


def _output(name: str, t: Optional[torch.Tensor], like: torch.Tensor, rows: int, cols: int):
    """The output of `like`'s shape, type and device (given or new): (it, its
    leading dimension)."""
    if t is None:
        return torch.empty((rows, cols), dtype=like.dtype, device=like.device), cols
    _need(t.dtype == like.dtype, f"{name} must be {like.dtype}, got {t.dtype}")
    return t, _matrix(name, t, like.get_device(), rows, cols)[2]


def _w_dtype(weight, bias) -> int:
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError(f"weight and bias differ in type: {weight.dtype}, {bias.dtype}")
    t = weight if weight is not None else bias
    return _lib.MUON_F32 if t is None else _dtype("weight and bias", t)


def _norm_forward(x, weight, bias, eps, out, keep, saved):
    """(y, mean, rstd, saved): with keep, h goes to a checkpoint and no mean
    is written."""
    rows, cols, ld, index = _matrix("x", x)
    dev = x.device
    y, ld_y = _output("out", out, x, rows, cols)
    rstd = torch.empty(rows, dtype=_F32, device=dev)
    if keep:
        saved = _checkpoint("saved", saved, rows, cols, x)
        mean, mean_at, fields = None, 0, saved._fields()
    else:
        mean = torch.empty(rows, dtype=_F32, device=dev)
        mean_at, fields = mean.data_ptr(), _NO_CKPT
    _call(index, "muon_layer_norm", _norm_args(
        x.data_ptr(), _vector("weight", weight, index, cols), _vector("bias", bias, index, cols),
        y.data_ptr(), mean_at, rstd.data_ptr(), *fields, rows, cols, ld, ld_y, _dtype("x", x),
        _w_dtype(weight, bias), eps))
    return y, mean, rstd, saved


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5,
               out: Optional[torch.Tensor] = None):
    """y = (x - mean) * rstd * weight + bias over the rows of x.

    Returns (y, mean, rstd); y has x's type (out may be x), mean and rstd are
    fp32.  weight and bias: fp32 or bf16, of one type; None for ones, zeros."""
    return _norm_forward(x, weight, bias, eps, out, False, None)[:3]


def layer_norm_checkpoint(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                          bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5,
                          out: Optional[torch.Tensor] = None,
                          saved: Optional[Checkpoint8] = None):
    """layer_norm that keeps h = (x - mean) * rstd as an 8-bit checkpoint, in
    the same pass.

    Returns (y, rstd, saved).  saved serves :func:`layer_norm_backward` and,
    with the norm's weight and bias, :func:`weight_grad` of every product that
    reads y, so that neither x nor y has to be kept."""
    y, _, rstd, saved = _norm_forward(x, weight, bias, eps, out, True, saved)
    return y, rstd, saved


def layer_norm_backward(dy: torch.Tensor, x, mean: Optional[torch.Tensor], rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None,
                        bias: Optional[torch.Tensor] = None, *,
                        out: Optional[torch.Tensor] = None):
    """The gradients of layer_norm: (dx, dweight, dbias).

    x: the forward pass's input with its mean, or the Checkpoint8 that
    layer_norm_checkpoint kept (mean is then None).  dweight and dbias have
    the types of weight and bias and are None where those are.  dx has dy's
    type (out may be dy)."""
    rows, cols, ld_dy, index = _matrix("dy", dy)
    dev = dy.device
    if isinstance(x, Checkpoint8):
        _need(x.shape == (rows, cols) and x.device == dev,
              f"x must be a checkpoint of {(rows, cols)} on {dev}, is of {x.shape}")
        _need(mean is None, "mean must be None beside a checkpoint (it holds h itself)")
        saved, x_ptr, ld_x = x._fields(), 0, 0
    else:
        ld_x = _matrix("x", x, index, rows, cols)[2]
        _need(x.dtype == dy.dtype, f"x and dy differ in type: {x.dtype}, {dy.dtype}")
        _need(mean is not None, "mean is needed beside x")
        saved, x_ptr = _NO_CKPT, x.data_ptr()
    dx, ld_dx = _output("out", out, dy, rows, cols)
    dw = db = None
    w_at = dw_at = db_at = 0
    if weight is not None:
        w_at = _vector("weight", weight, index, cols)
        dw = torch.empty(cols, dtype=weight.dtype, device=dev)
        dw_at = dw.data_ptr()
    if bias is not None:
        _vector("bias", bias, index, cols)
        db = torch.empty(cols, dtype=bias.dtype, device=dev)
        db_at = db.data_ptr()
    _call_ws(index, "muon_layer_norm_grad", "muon_layer_norm_grad_workspace", _norm_grad_args(
        dy.data_ptr(), x_ptr, _vector("mean", mean, index, rows, _F32),
        _vector("rstd", rstd, index, rows, _F32), w_at, dx.data_ptr(), dw_at, db_at,
        *saved, rows, cols, ld_dy, ld_x, ld_dx, _dtype("dy", dy), _w_dtype(weight, bias)), dev)
    return dx, dw, db


def _gradient(name: str, t: torch.Tensor, shape, index: int):
    """Checks a row-major gradient (n x k, or experts x n x k): (ld, stride)."""
    if t.shape != shape or t.get_device() != index:
        raise ValueError(f"{name} must be {shape} on cuda:{index}, got {tuple(t.shape)} on {t.device}")
    if t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be row-major (stride(-1) == 1)")
    return t.stride(-2), t.stride(0) if len(shape) == 3 else 0


def weight_grad(dy: torch.Tensor, x: Checkpoint8, *, weight: Optional[torch.Tensor] = None,
                bias: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                add: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The gradient of W (n x k) of a product Y = X W^T: dY^T X (+ add).

    dy: tokens x n, bf16.  x: the checkpoint of X, or of the h of the norm
    that X came from, with that norm's weight and bias (k values each, fp32 or
    bf16, of one type).
    offsets: experts + 1 int32 values on the device; the result is then
    experts x n x k, matrix e over the tokens offsets[e] .. offsets[e + 1].
    add may be out (gradient accumulation).  out (or a new tensor of dtype):
    fp32 or bf16; the matrices of a Muon set's gradients can be given."""
    rows, n, ld_dy, index = _matrix("dy", dy)
    _need(dy.dtype == _BF16, f"dy must be bfloat16, got {dy.dtype}")
    k, dev = x.cols, dy.device
    _need(x.q.shape[0] == rows and x.q.get_device() == index,
          f"x must hold {rows} rows on {dev}, has {x.rows} on {x.device}")
    experts, offsets_at, shape = 1, 0, (n, k)
    if offsets is not None:
        _need(offsets.dim() == 1 and offsets.shape[0] >= 2, "offsets must be experts + 1 values")
        experts = offsets.shape[0] - 1
        offsets_at = _vector("offsets", offsets, index, experts + 1, _I32)
        shape = (experts, n, k)
    if out is None:
        g = torch.empty(shape, dtype=dtype, device=dev)
        ld_g, stride_g = k, n * k
    else:
        g = out
        ld_g, stride_g = _gradient("out", g, shape, index)
    ld_c = stride_c = add_at = 0
    if add is not None:
        ld_c, stride_c = _gradient("add", add, shape, index)
        _need(add.dtype == g.dtype, f"add and the result differ in type: {add.dtype}, {g.dtype}")
        add_at = add.data_ptr()
    _call_ws(index, "muon_weight_grad", "muon_weight_grad_workspace", _weight_grad_args(
        dy.data_ptr(), _vector("weight", weight, index, k), _vector("bias", bias, index, k), add_at,
        g.data_ptr(), offsets_at, *x._fields(), rows, n, k, experts, ld_dy, ld_c, ld_g, stride_c,
        stride_g, _dtype("out", g), _w_dtype(weight, bias)), dev)
    return g


class Routing:
    """What :func:`route` gives: indices (int32) and weights (fp32), tokens x
    k; counts (int32) per expert and their running sum offsets (experts + 1);
    loss (fp32) and kept (int32, the tokens that took part), one value each;
    and the settings that the backward pass needs again."""

    __slots__ = ("indices", "weights", "counts", "kept", "offsets", "loss", "coef", "renormalise")

    def __init__(self, indices, weights, counts, kept, *, offsets=None, loss=None,
                 coef: float = 0.01, renormalise: bool = True):
        self.indices, self.weights, self.counts, self.kept = indices, weights, counts, kept
        self.offsets, self.loss, self.coef, self.renormalise = offsets, loss, coef, renormalise


def route(logits: torch.Tensor, k: int, *, mask: Optional[torch.Tensor] = None,
          coef: float = 0.01, renormalise: bool = True) -> Routing:
    """The router of a mixture-of-experts block over logits (tokens x
    experts, fp32 or bf16): the k largest of every token, their softmax
    weights, counts per expert and the balance loss times coef.
    mask (bool or uint8, one per token): tokens with 0 take no part."""
    tokens, experts, ld, index = _matrix("logits", logits)
    dev = logits.device
    mask_at = 0
    if mask is not None:
        _need(mask.dtype in (torch.bool, torch.uint8), f"mask must be bool or uint8, got {mask.dtype}")
        mask_at = _vector("mask", mask, index, tokens)
    if not 1 <= k <= min(experts, 32):
        raise ValueError(f"k must be 1 .. min(experts, 32), got {k}")
    indices = torch.empty((tokens, k), dtype=_I32, device=dev)
    weights = torch.empty((tokens, k), dtype=_F32, device=dev)
    counts = torch.empty(experts, dtype=_I32, device=dev)
    offsets = torch.empty(experts + 1, dtype=_I32, device=dev)
    kept = torch.empty((), dtype=_I32, device=dev)
    loss = torch.empty((), dtype=_F32, device=dev)
    _call_ws(index, "muon_route", "muon_route_workspace", _route_args(
        logits.data_ptr(), mask_at, indices.data_ptr(), weights.data_ptr(), counts.data_ptr(),
        offsets.data_ptr(), loss.data_ptr(), kept.data_ptr(), tokens, experts, k, ld,
        _dtype("logits", logits), bool(renormalise), coef), dev)
    return Routing(indices, weights, counts, kept, offsets=offsets, loss=loss, coef=coef,
                   renormalise=renormalise)


def route_backward(logits: torch.Tensor, routing: Routing, *,
                   dloss: Optional[torch.Tensor] = None,
                   dweights: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient with respect to the logits, from that of the loss (one
    fp32 value on the device) and of the weights (tokens x k, fp32).  Returns
    dlogits of the logits' type (out may be logits)."""
    tokens, experts, ld, index = _matrix("logits", logits)
    r = routing
    indices, weights, counts = r.indices, r.weights, r.counts
    _need(indices.dim() == 2, "routing.indices must be 2-D")
    k = indices.shape[1]
    if (indices.dtype != _I32 or weights.dtype != _F32 or counts.dtype != _I32
            or indices.shape[0] != tokens or weights.shape != (tokens, k)
            or counts.shape != (experts,) or r.kept.dtype != _I32 or r.kept.numel() != 1
            or not (indices.is_contiguous() and weights.is_contiguous() and counts.is_contiguous())
            or not (indices.get_device() == weights.get_device() == counts.get_device()
                    == r.kept.get_device() == index)):
        raise ValueError(f"routing does not belong to logits of {(tokens, experts)} on "
                         f"{logits.device} (dense int32 indices and fp32 weights of tokens x k, "
                         "int32 counts of the experts and kept)")
    dloss_at = dweights_at = ld_dw = 0
    if dloss is not None:
        if dloss.dtype != _F32 or dloss.numel() != 1 or dloss.get_device() != index:
            raise ValueError("dloss must be one float32 value on the device")
        dloss_at = dloss.data_ptr()
    if dweights is not None:
        ld_dw = _matrix("dweights", dweights, index, tokens, k)[2]
        _need(dweights.dtype == _F32, f"dweights must be float32, got {dweights.dtype}")
        dweights_at = dweights.data_ptr()
    dz, ld_dz = _output("out", out, logits, tokens, experts)
    _call(index, "muon_route_grad", _route_grad_args(
        logits.data_ptr(), indices.data_ptr(), weights.data_ptr(), counts.data_ptr(),
        r.kept.data_ptr(), dloss_at, dweights_at, dz.data_ptr(), tokens, experts, k, ld, ld_dw,
        ld_dz, _dtype("logits", logits), bool(r.renormalise), r.coef))
    return dz


def ops_sync(device: Optional[int] = None) -> None:
    """Waits for the current stream and raises what the operators met on the
    GPU (MuonError; a bounded wait that ran out is MUON_ERR_TIMEOUT)."""
    _call(torch.cuda.current_device() if device is None else device, "muon_ops_sync")
