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


def _need(ok: bool, message: str) -> None:
    if not ok:
        raise ValueError(message)


def _dtype(name: str, t: torch.Tensor) -> int:
    d = _DT.get(t.dtype)
    if d is None:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return d


def _matrix(name: str, t: torch.Tensor, device=None, shape=None) -> int:
    """Checks a row-major 2-D CUDA tensor; its leading dimension."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(t.shape)}")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a CUDA tensor of its operator's device, is on {t.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    ld, inner = t.stride()
    if inner != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must be row-major (stride(1) == 1)")
    return ld


def _vector(name: str, t: Optional[torch.Tensor], device, n: int, dtype=None) -> int:
    """Checks a dense 1-D tensor of n values (or None); its address."""
    if t is None:
        return 0
    if t.device != device or t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be {n} dense values on {device}, got {tuple(t.shape)} "
                         f"on {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _call(device: torch.device, name: str, *args) -> None:
    """Calls an entry point on the device's current stream, with the device
    current."""
    index = device.index
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return _call(device, name, *args)
    err = _local.err
    rc = getattr(lib(), name)(*args, torch._C._cuda_getCurrentRawStream(index), err, _ERR_LEN)
    if rc < 0:
        raise MuonError(rc, f"{name}: {err.value.decode(errors='replace')}")


def _call_ws(device: torch.device, name: str, query: str, args: bytes) -> None:
    """Calls an entry point that takes a workspace, allocated here."""
    size = _local.size
    size.value = 0
    # a query that refuses its arguments leaves the message to the call
    getattr(lib(), query)(args, _local.size_ref)
    n = size.value
    if n:
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        _call(device, name, args, ws.data_ptr(), n)
    else:
        _call(device, name, args, None, 0)


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
        rows, dev = q.shape[0], q.device
        if out is None:
            out = torch.empty((rows, cols), dtype=dtype, device=dev)
        ld = _matrix("out", out, dev, (rows, cols))
        _call(dev, "muon_ckpt8_unpack", _ckpt_arg(*self._fields()), rows, cols, out.data_ptr(),
              _dtype("out", out), ld)
        return out


def checkpoint8(x: torch.Tensor, out: Optional[Checkpoint8] = None) -> Checkpoint8:
    """The 8-bit checkpoint of x (2-D, fp32 or bf16)."""
    ld = _matrix("x", x)
    rows, cols = x.shape
    dev = x.device
    out = _checkpoint("out", out, rows, cols, dev)
    _call(dev, "muon_ckpt8_pack", x.data_ptr(), _dtype("x", x), rows, cols, ld,
          _ckpt_arg(*out._fields()))
    return out


def _checkpoint(name: str, c: Optional[Checkpoint8], rows: int, cols: int, device) -> Checkpoint8:
    if c is None:
        return Checkpoint8.empty(rows, cols, device)
    _need(c.shape == (rows, cols) and c.device == device,
          f"{name} must be a checkpoint of {(rows, cols)} on {device}")
    return c


def _output(name: str, t: Optional[torch.Tensor], like: torch.Tensor):
    """The output of `like`'s shape, type and device (given or new): (it, its
    leading dimension)."""
    if t is None:
        rows, cols = like.shape
        return torch.empty((rows, cols), dtype=like.dtype, device=like.device), cols
    _need(t.dtype == like.dtype, f"{name} must be {like.dtype}, got {t.dtype}")
    return t, _matrix(name, t, like.device, like.shape)


def _w_dtype(weight, bias) -> int:
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError(f"weight and bias differ in type: {weight.dtype}, {bias.dtype}")
    t = weight if weight is not None else bias
    return _lib.MUON_F32 if t is None else _dtype("weight and bias", t)


def _norm_forward(x, weight, bias, eps, out, saved, mean):
    ld = _matrix("x", x)
    rows, cols = x.shape
    dev = x.device
    y, ld_y = _output("out", out, x)
    rstd = torch.empty(rows, dtype=_F32, device=dev)
    args = _norm_args(
        x.data_ptr(), _vector("weight", weight, dev, cols), _vector("bias", bias, dev, cols),
        y.data_ptr(), 0 if mean is None else mean.data_ptr(), rstd.data_ptr(),
        *(_NO_CKPT if saved is None else saved._fields()),
        rows, cols, ld, ld_y, _dtype("x", x), _w_dtype(weight, bias), eps)
    _call(dev, "muon_layer_norm", args)
    return y, rstd


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5,
               out: Optional[torch.Tensor] = None):
    """y = (x - mean) * rstd * weight + bias over the rows of x.

    Returns (y, mean, rstd); y has x's type (out may be x), mean and rstd are
    fp32.  weight and bias: fp32 or bf16, of one type; None for ones, zeros."""
    _matrix("x", x)
    mean = torch.empty(x.shape[0], dtype=_F32, device=x.device)
    y, rstd = _norm_forward(x, weight, bias, eps, out, None, mean)
    return y, mean, rstd


def layer_norm_checkpoint(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                          bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5,
                          out: Optional[torch.Tensor] = None,
                          saved: Optional[Checkpoint8] = None):
    """layer_norm that keeps h = (x - mean) * rstd as an 8-bit checkpoint, in
    the same pass.

    Returns (y, rstd, saved).  saved serves :func:`layer_norm_backward` and,
    with the norm's weight and bias, :func:`weight_grad` of every product that
    reads y, so that neither x nor y has to be kept."""
    _matrix("x", x)
    saved = _checkpoint("saved", saved, x.shape[0], x.shape[1], x.device)
    y, rstd = _norm_forward(x, weight, bias, eps, out, saved, None)
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
    ld_dy = _matrix("dy", dy)
    rows, cols = dy.shape
    dev = dy.device
    if isinstance(x, Checkpoint8):
        _need(x.shape == (rows, cols) and x.device == dev,
              f"x must be a checkpoint of {(rows, cols)} on {dev}, is of {x.shape}")
        _need(mean is None, "mean must be None beside a checkpoint (it holds h itself)")
        saved, x_ptr, ld_x = x._fields(), 0, 0
    else:
        ld_x = _matrix("x", x, dev, dy.shape)
        _need(x.dtype == dy.dtype, f"x and dy differ in type: {x.dtype}, {dy.dtype}")
        _need(mean is not None, "mean is needed beside x")
        saved, x_ptr = _NO_CKPT, x.data_ptr()
    dx, ld_dx = _output("out", out, dy)
    dw = torch.empty(cols, dtype=weight.dtype, device=dev) if weight is not None else None
    db = torch.empty(cols, dtype=bias.dtype, device=dev) if bias is not None else None
    _vector("bias", bias, dev, cols)
    args = _norm_grad_args(
        dy.data_ptr(), x_ptr, _vector("mean", mean, dev, rows, _F32),
        _vector("rstd", rstd, dev, rows, _F32), _vector("weight", weight, dev, cols),
        dx.data_ptr(), 0 if dw is None else dw.data_ptr(), 0 if db is None else db.data_ptr(),
        *saved, rows, cols, ld_dy, ld_x, ld_dx, _dtype("dy", dy), _w_dtype(weight, bias))
    _call_ws(dev, "muon_layer_norm_grad", "muon_layer_norm_grad_workspace", args)
    return dx, dw, db


def _gradient(name: str, t: torch.Tensor, shape, device):
    """Checks a row-major gradient (n x k, or experts x n x k): (ld, stride)."""
    if t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be {shape} on {device}, got {tuple(t.shape)} on {t.device}")
    if t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be row-major (stride(-1) == 1)")
    return t.stride(-2), t.stride(0) if len(shape) == 3 else 0


def weight_grad(dy: torch.Tensor, x: Checkpoint8, *, weight: Optional[torch.Tensor] = None,
                bias: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                add: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The gradient of W (n x k) of a product Y = X W^T: dY^T X (+ add).

    dy: tokens x n, bf16.  x: the checkpoint of X, or of the h of the norm
    that X came from, with that norm's weight and bias (k fp32 values each).
    offsets: experts + 1 int32 values on the device; the result is then
    experts x n x k, matrix e over the tokens offsets[e] .. offsets[e + 1].
    add may be out (gradient accumulation).  out (or a new tensor of dtype):
    fp32 or bf16; the matrices of a Muon set's gradients can be given."""
    ld_dy = _matrix("dy", dy)
    _need(dy.dtype == torch.bfloat16, f"dy must be bfloat16, got {dy.dtype}")
    rows, n = dy.shape
    k, dev = x.cols, dy.device
    _need(x.rows == rows and x.device == dev,
          f"x must hold {rows} rows on {dev}, has {x.rows} on {x.device}")
    experts = 1
    if offsets is not None:
        _need(offsets.dim() == 1 and offsets.shape[0] >= 2, "offsets must be experts + 1 values")
        experts = offsets.shape[0] - 1
        _vector("offsets", offsets, dev, experts + 1, torch.int32)
    shape = (n, k) if offsets is None else (experts, n, k)
    g = torch.empty(shape, dtype=dtype, device=dev) if out is None else out
    ld_g, stride_g = _gradient("out", g, shape, dev)
    ld_c = stride_c = 0
    if add is not None:
        ld_c, stride_c = _gradient("add", add, shape, dev)
        _need(add.dtype == g.dtype, f"add and the result differ in type: {add.dtype}, {g.dtype}")
    args = _weight_grad_args(
        dy.data_ptr(), _vector("weight", weight, dev, k, _F32),
        _vector("bias", bias, dev, k, _F32), 0 if add is None else add.data_ptr(),
        g.data_ptr(), 0 if offsets is None else offsets.data_ptr(), *x._fields(),
        rows, n, k, experts, ld_dy, ld_c, ld_g, stride_c, stride_g, _dtype("out", g))
    _call_ws(dev, "muon_weight_grad", "muon_weight_grad_workspace", args)
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
    ld = _matrix("logits", logits)
    tokens, experts = logits.shape
    dev = logits.device
    mask_ptr = 0
    if mask is not None:
        _need(mask.dtype in (torch.bool, torch.uint8), f"mask must be bool or uint8, got {mask.dtype}")
        mask_ptr = _vector("mask", mask, dev, tokens)
    _need(1 <= k <= min(experts, 32), f"k must be 1 .. min(experts, 32), got {k}")
    indices = torch.empty((tokens, k), dtype=_I32, device=dev)
    weights = torch.empty((tokens, k), dtype=_F32, device=dev)
    counts = torch.empty(experts, dtype=_I32, device=dev)
    offsets = torch.empty(experts + 1, dtype=_I32, device=dev)
    kept = torch.empty((), dtype=_I32, device=dev)
    loss = torch.empty((), dtype=_F32, device=dev)
    args = _route_args(
        logits.data_ptr(), mask_ptr, indices.data_ptr(), weights.data_ptr(), counts.data_ptr(),
        offsets.data_ptr(), loss.data_ptr(), kept.data_ptr(), tokens, experts, k, ld,
        _dtype("logits", logits), bool(renormalise), coef)
    _call_ws(dev, "muon_route", "muon_route_workspace", args)
    return Routing(indices, weights, counts, kept, offsets=offsets, loss=loss, coef=coef,
                   renormalise=renormalise)


def route_backward(logits: torch.Tensor, routing: Routing, *,
                   dloss: Optional[torch.Tensor] = None,
                   dweights: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient with respect to the logits, from that of the loss (one
    fp32 value on the device) and of the weights (tokens x k, fp32).  Returns
    dlogits of the logits' type (out may be logits)."""
    ld = _matrix("logits", logits)
    tokens, experts = logits.shape
    dev = logits.device
    r = routing
    _need(r.indices.dim() == 2, "routing.indices must be 2-D")
    k = r.indices.shape[1]
    for name, t, dtype, shape in (("indices", r.indices, _I32, (tokens, k)),
                                  ("weights", r.weights, _F32, (tokens, k)),
                                  ("counts", r.counts, _I32, (experts,))):
        if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != dev:
            raise ValueError(f"routing.{name} must be {dtype} {shape}, dense, on {dev}")
    _need(r.kept.dtype == _I32 and r.kept.numel() == 1 and r.kept.device == dev,
          "routing.kept must be one int32 value on the device")
    if dloss is not None:
        _need(dloss.dtype == _F32 and dloss.numel() == 1 and dloss.device == dev,
              "dloss must be one float32 value on the device")
    ld_dw = 0
    if dweights is not None:
        ld_dw = _matrix("dweights", dweights, dev, (tokens, k))
        _need(dweights.dtype == torch.float32, f"dweights must be float32, got {dweights.dtype}")
    dz, ld_dz = _output("out", out, logits)
    args = _route_grad_args(
        logits.data_ptr(), r.indices.data_ptr(), r.weights.data_ptr(), r.counts.data_ptr(),
        r.kept.data_ptr(), 0 if dloss is None else dloss.data_ptr(),
        0 if dweights is None else dweights.data_ptr(), dz.data_ptr(), tokens, experts, k,
        ld, ld_dw, ld_dz, _dtype("logits", logits), bool(r.renormalise), r.coef)
    _call(dev, "muon_route_grad", args)
    return dz


def ops_sync(device: Optional[int] = None) -> None:
    """Waits for the current stream and raises what the operators met on the
    GPU (MuonError; a bounded wait that ran out is MUON_ERR_TIMEOUT)."""
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
    _call(dev, "muon_ops_sync")
