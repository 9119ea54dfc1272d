"""Python face of libmuon's operators inside a block: the gated feed-forward
block (dense, or one per expert over a router's offsets), rotary positions of
queries and keys, and dropout, each with its backward pass.

    q, k = rotary(q, k, plan)                                 # plan = RotaryPlan(head_dim)
    ...
    x = dropout(attention, p, seed, step, residual=x)
    y, saved = gated_ffn(rows, w_gate, w_up, w_down, offsets=r.offsets)
    drows, dw_gate, dw_up, dw_down = gated_ffn_backward(dy, rows, saved, w_gate, w_up, w_down,
                                                        offsets=r.offsets)

They keep to :mod:`~newton_schulz_06_gb300.ops`: work is queued on the current
stream of the tensors' device, outputs that are not given are allocated,
nothing records for torch.autograd, and the same call gives the same bits
again.  include/muon.h has the formulas.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import Optional, Tuple, Union

import torch

from . import _lib
from ._lib import MuonError
from .ops import (_BF16, _ERR_LEN, _I32, _call, _call_ws, _dtype, _fn, _gradient, _local,
                  _matrix, _need, _output, _vector, Checkpoint8, weight_grad)
from .muon import _DT

_ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
_ffn_args = _lib.packer(_lib.GatedFfnArgs).pack
_ffn_grad_args = _lib.packer(_lib.GatedFfnGradArgs).pack
_rotary_args = _lib.packer(_lib.RotaryArgs).pack
_dropout_args = _lib.packer(_lib.DropoutArgs).pack
_NO_TENSOR = (0, 0, 0, 0, 0, 0, 0, 0, 0)


# ------------------------------------------------------- gated feed-forward

def _rows(name: str, t: torch.Tensor, index: int = -1, rows: int = -1, cols: int = -1):
    """_matrix of a bf16 tensor."""
    if t.dtype != _BF16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    return _matrix(name, t, index, rows, cols)


def _experts(offsets: Optional[torch.Tensor], index: int) -> Tuple[int, int]:
    """(experts, or 0 for a dense block; address of the offsets)."""
    if offsets is None:
        return 0, 0
    _need(offsets.dim() == 1 and offsets.shape[0] >= 2, "offsets must be experts + 1 values")
    experts = offsets.shape[0] - 1
    return experts, _vector("offsets", offsets, index, experts + 1, _I32)


def _weight(name: str, w: torch.Tensor, shape: tuple, index: int):
    """Checks a bf16 matrix, or experts x a matrix: (leading dimension, stride)."""
    if w.dtype != _BF16:
        raise ValueError(f"{name} must be bfloat16, got {w.dtype}")
    if w.shape != shape or w.get_device() != index:
        raise ValueError(f"{name} must be {shape} on cuda:{index}, got {tuple(w.shape)} on {w.device}")
    stride = w.stride()
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be row-major (stride(-1) == 1)")
    return stride[-2], stride[0] if len(shape) == 3 else 0


def _weights(index: int, experts: int, hidden: int, gate, up, down):
    """Checks the three matrices (or experts x matrices); (inner, the shapes of
    gate and up and of down, their leading dimensions, their strides)."""
    shape = gate.shape
    if len(shape) != (3 if experts else 2):
        raise ValueError(f"w_gate must be {'experts x inner x hidden' if experts else 'inner x hidden'}, "
                         f"got {tuple(shape)}")
    inner = shape[-2]
    if experts:
        one, two = (experts, inner, hidden), (experts, hidden, inner)
    else:
        one, two = (inner, hidden), (hidden, inner)
    ld_gate, stride_gate = _weight("w_gate", gate, one, index)
    ld_up, stride_up = _weight("w_up", up, one, index)
    ld_down, stride_down = _weight("w_down", down, two, index)
    return inner, one, two, (ld_gate, ld_up, ld_down), (stride_gate, stride_up, stride_down)


def _activation(name: str) -> int:
    code = _ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}, got {name!r}")
    return code


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, *,
              offsets: Optional[torch.Tensor] = None, activation: str = "silu", keep: bool = True,
              out: Optional[torch.Tensor] = None):
    """y = (act(x w_gate^T) * (x w_up^T)) w_down^T, in bf16 with fp32 sums.

    x: rows x hidden; w_gate, w_up: inner x hidden; w_down: hidden x inner.
    offsets (experts + 1 int32 values on the device, e.g. Routing.offsets): x
    holds the rows by expert, and the weights are experts x matrices; rows of
    no expert are not written (a new y holds anything there).
    activation: "silu", "gelu" (by erf) or "gelu_tanh".
    Returns (y, saved): saved is (g, u), both rows x inner, for
    :func:`gated_ffn_backward`, or None without keep.  They are rounded to
    bf16, which is half of the squared error that the gradients then have.  out
    may be x.
    The last bits of a row may depend on the number of rows beside it (long sums
    of few rows are added up in parts)."""
    rows, hidden, ld_x, index = _rows("x", x)
    act = _activation(activation)
    experts, offsets_at = _experts(offsets, index)
    inner, _, _, lds, strides = _weights(index, experts, hidden, w_gate, w_up, w_down)
    y, ld_y = _output("out", out, x, rows, hidden)
    saved, gate_at, up_at, dev = None, 0, 0, x.device
    if keep:
        gate = torch.empty((rows, inner), dtype=_BF16, device=dev)
        up = torch.empty((rows, inner), dtype=_BF16, device=dev)
        saved, gate_at, up_at = (gate, up), gate.data_ptr(), up.data_ptr()
    _call_ws(index, "muon_gated_ffn", "muon_gated_ffn_workspace", _ffn_args(
        x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), y.data_ptr(), gate_at, up_at,
        offsets_at, rows, hidden, inner, experts or 1, ld_x, *lds, ld_y, inner, *strides, act), dev)
    return y, saved


def gated_ffn_backward(dy: torch.Tensor, x: Union[torch.Tensor, Checkpoint8, None], saved,
                       w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, *,
                       offsets: Optional[torch.Tensor] = None, activation: str = "silu",
                       weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, grads=None, accumulate: bool = False,
                       dtype: torch.dtype = _BF16):
    """The gradients of gated_ffn: (dx, dw_gate, dw_up, dw_down).

    saved: what gated_ffn kept.  x: its input, or a Checkpoint8 of it, or of the
    h of a norm that made it (weight, bias: that norm's); None leaves out the
    gradients of w_gate and w_up.
    grads: (dw_gate, dw_up, dw_down) to write, fp32 or bf16 tensors of the
    weights' shapes, e.g. those that a Muon set steps with (new ones of dtype
    otherwise); with accumulate the gradients are added to them.  Experts
    without rows get zeros.  out: receives dx (it may not share memory with dy or x)."""
    rows, hidden, ld_dy, index = _rows("dy", dy)
    dev = dy.device
    act = _activation(activation)
    experts, offsets_at = _experts(offsets, index)
    inner, one, two, lds, strides = _weights(index, experts, hidden, w_gate, w_up, w_down)
    gate, up = saved
    ld_kept = _rows("gate", gate, index, rows, inner)[2]
    if _rows("up", up, index, rows, inner)[2] != ld_kept and rows > 1:
        raise ValueError("gate and up differ in their strides")
    checkpoint = isinstance(x, Checkpoint8)
    ld_x = x_at = 0
    if checkpoint:
        _need(x.shape == (rows, hidden) and x.device == dev,
              f"x must be a checkpoint of {(rows, hidden)} on {dev}, is of {x.shape}")
    else:
        _need(weight is None and bias is None, "weight and bias go with a checkpoint of x")
        if x is not None:
            ld_x, x_at = _rows("x", x, index, rows, hidden)[2], x.data_ptr()
    dx, ld_dx = _output("out", out, dy, rows, hidden)
    dx_at, dy_at = dx.data_ptr(), dy.data_ptr()
    if out is not None and rows and (dx_at == dy_at or dx_at == x_at):
        raise ValueError("out may not be dy or x: they are read after it is written")
    if grads is None:
        _need(not accumulate, "accumulate needs grads to add to")
        code = _DT.get(dtype)
        _need(code is not None, f"dtype must be float32 or bfloat16, got {dtype}")
        dg = du = None
        if x is not None:
            dg, du = torch.empty(one, dtype=dtype, device=dev), torch.empty(one, dtype=dtype, device=dev)
        dd = torch.empty(two, dtype=dtype, device=dev)
        ld_g, size = (hidden, hidden, inner), inner * hidden
        stride_g = (size, size, size)
    else:
        dg, du, dd = grads
        if x is None:
            dg = du = None
        kind = next((g.dtype for g in (dg, du, dd) if g is not None), _BF16)
        code = _DT.get(kind)
        _need(code is not None, f"grads must be float32 or bfloat16, got {kind}")
        ld_g, stride_g = [0, 0, 0], [0, 0, 0]
        for i, (name, g, shape) in enumerate((("dw_gate", dg, one), ("dw_up", du, one), ("dw_down", dd, two))):
            if g is not None:
                ld_g[i], stride_g[i] = _gradient(name, g, shape, index)
                _need(g.dtype == kind, "grads differ in type")
    dgate = dup = None
    dgate_at = dup_at = ld_d = 0
    if checkpoint:
        dgate = torch.empty((rows, inner), dtype=_BF16, device=dev)
        dup = torch.empty((rows, inner), dtype=_BF16, device=dev)
        dgate_at, dup_at, ld_d = dgate.data_ptr(), dup.data_ptr(), inner
    _call_ws(index, "muon_gated_ffn_grad", "muon_gated_ffn_grad_workspace", _ffn_grad_args(
        dy_at, x_at, gate.data_ptr(), up.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
        dx_at, 0 if checkpoint or dg is None else dg.data_ptr(), 0 if checkpoint or du is None else du.data_ptr(),
        0 if dd is None else dd.data_ptr(), dgate_at, dup_at, 0, offsets_at, rows, hidden, inner, experts or 1,
        ld_dy, ld_x, ld_kept, *lds, ld_dx, ld_d, *ld_g, *strides, *stride_g, act, code, bool(accumulate)), dev)
    if checkpoint:
        for d, g in ((dgate, dg), (dup, du)):
            if g is not None:
                weight_grad(d, x, weight=weight, bias=bias, offsets=offsets, add=g if accumulate else None, out=g)
    return dx, dg, du, dd


# --------------------------------------------------------- rotary positions

class RotaryPlan:
    """The frequencies of a rotary embedding of the first `dim` values of a
    head (even, at most 512): pair i turns by base^(-2 i / dim) radians a
    position.

    layout: "half" (value i with i + dim / 2) or "interleaved" (2 i with 2 i + 1).
    scaling, for contexts longer than the trained one: "none", "linear"
    (frequencies divided by factor), "ntk" (a larger base) or "yarn" (divided
    for the pairs that turn less than slow times in `original` positions, kept
    for those that turn more than fast times, a ramp between, and the result
    times 0.1 ln(factor) + 1).  A plan is host data and serves any device."""

    __slots__ = ("dim", "layout", "scale", "_turns")

    def __init__(self, dim: int, *, base: float = 10000.0, layout: str = "half", scaling: str = "none",
                 factor: float = 1.0, original: float = 4096, fast: float = 32.0, slow: float = 1.0):
        _need(dim % 2 == 0 and 2 <= dim <= 512, f"dim must be even and 2 .. 512, got {dim}")
        if layout not in _LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
        if scaling not in _SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}, got {scaling!r}")
        turns, scale = (ctypes.c_uint64 * (dim // 2))(), ctypes.c_float()
        err = _local.err
        rc = _fn("muon_rotary_frequencies")(dim // 2, base, _SCALINGS[scaling], factor, original, fast, slow,
                                            turns, ctypes.byref(scale), err, _ERR_LEN)
        if rc < 0:
            raise MuonError(rc, f"muon_rotary_frequencies: {err.value.decode(errors='replace')}")
        self.dim, self.layout, self.scale = dim, _LAYOUTS[layout], scale.value
        self._turns = bytes(turns)       # one 64-bit fraction of a turn a pair

    @property
    def frequencies(self) -> Tuple[float, ...]:
        """Radians a position of every pair."""
        return tuple(t * (2.0 * math.pi) * 2.0 ** -64
                     for t in struct.unpack(f"={self.dim // 2}Q", self._turns))


def _heads(name: str, t: torch.Tensor, index: int):
    """Checks a tensor of (batch x) seq x heads x head: (its shape with a batch,
    its strides of batch, seq and heads)."""
    shape, strides = t.shape, t.stride()
    n = len(shape)
    if n != 4 and n != 3:
        raise ValueError(f"{name} must be seq x heads x head, or batch x seq x heads x head, got "
                         f"{tuple(shape)}")
    on = t.get_device()
    if on < 0 or on != index:
        raise ValueError(f"{name} must be a CUDA tensor of its operator's device, is on {t.device}")
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}'s heads must be dense (stride(-1) == 1)")
    if n == 3:
        return (1, *shape), (0, strides[0], strides[1])
    return shape, strides[:3]


def _turned(name: str, x: torch.Tensor, out, shape, strides, index: int):
    """(the C argument of one tensor, its output: given or new)."""
    batch, seq, heads, head = shape
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        row = heads * head
        to = (seq * row, row, head)
    else:
        if out.dtype != x.dtype or out.shape != x.shape:
            raise ValueError(f"out_{name} must be {tuple(x.shape)} of {x.dtype}, got {tuple(out.shape)} of "
                             f"{out.dtype}")
        to = _heads(f"out_{name}", out, index)[1]
        for n, stride in zip(shape, to):
            _need(stride > 0 or n <= 1, f"out_{name} has places that share memory")
    return (x.data_ptr(), out.data_ptr(), heads, *strides, *to), out


def _address(b: bytes) -> int:
    """Where an object's bytes are, for a call that reads them before it returns."""
    return ctypes.cast(b, ctypes.c_void_p).value


def _turn(q, k, plan: RotaryPlan, positions, offset: int, out_q, out_k, inverse: bool):
    index = q.get_device()
    shape, strides = _heads("q", q, index)
    batch, seq, _, head = shape
    dtype = _dtype("q", q)
    if not -(1 << 63) <= offset < 1 << 63:
        raise ValueError(f"offset must be a 64-bit whole number, got {offset}")
    if plan.dim > head:
        raise ValueError(f"heads of {head} values are shorter than the plan's {plan.dim}")
    first, out_q = _turned("q", q, out_q, shape, strides, index)
    second = _NO_TENSOR
    if k is not None:
        shape_k, strides = _heads("k", k, index)
        if k.dtype != q.dtype or shape_k[0] != batch or shape_k[1] != seq or shape_k[3] != head \
                or k.dim() != q.dim():
            raise ValueError(f"k must match q in all but its heads, got {tuple(k.shape)} of {k.dtype}")
        second, out_k = _turned("k", k, out_k, shape_k, strides, index)
    else:
        _need(out_k is None, "out_k without k")
    at = stride = wide = 0
    if positions is not None:
        if positions.dtype not in (_I32, torch.int64):
            raise ValueError(f"positions must be int32 or int64, got {positions.dtype}")
        _need(positions.get_device() == index, f"positions must be on {q.device}")
        want = tuple(positions.shape)
        _need(want in ((seq,), (1, seq), (batch, seq)),
              f"positions must be {(seq,)} or {(batch, seq)}, got {want}")
        _need(positions.stride(-1) == 1 or seq <= 1, "positions must be dense along seq")
        at, wide = positions.data_ptr(), positions.dtype == torch.int64
        stride = positions.stride(0) if len(want) == 2 and want[0] > 1 else 0
    _call(index, "muon_rotary", _rotary_args(
        *first, *second, at, _address(plan._turns), batch, seq, head, plan.dim // 2, stride, offset, dtype,
        plan.layout, wide, inverse, plan.scale))
    return out_q, out_k


def rotary(q: torch.Tensor, k: Optional[torch.Tensor], plan: RotaryPlan, *,
           positions: Optional[torch.Tensor] = None, offset: int = 0,
           out_q: Optional[torch.Tensor] = None, out_k: Optional[torch.Tensor] = None):
    """Turns the first plan.dim values of every head of q and k (or of q alone)
    by their positions; the others are copied.  Returns (q', k').

    q, k: seq x heads x head, or batch x seq x heads x head, fp32 or bf16; any
    strides but that a head is dense, so that views (a transposed batch, the
    last values of longer heads) do.  out_q, out_k may be q and k themselves, and
    otherwise share no memory with either.
    positions: int32 or int64, seq or batch x seq; None counts from 0.  offset
    is added to each."""
    return _turn(q, k, plan, positions, offset, out_q, out_k, False)


def rotary_backward(dq: torch.Tensor, dk: Optional[torch.Tensor], plan: RotaryPlan, *,
                    positions: Optional[torch.Tensor] = None, offset: int = 0,
                    out_q: Optional[torch.Tensor] = None, out_k: Optional[torch.Tensor] = None):
    """The gradients of rotary's q and k from those of its results."""
    return _turn(dq, dk, plan, positions, offset, out_q, out_k, True)


# ----------------------------------------------------------------- dropout

_U64 = (1 << 64) - 1


def _drop(name, x, p, seed, offset, counter, residual, out):
    rows, cols, ld, index = _matrix(name, x)
    y, ld_y = _output("out", out, x, rows, cols)
    r_at = ld_r = counter_at = 0
    if residual is not None:
        _need(residual.dtype == x.dtype, f"residual must be {x.dtype}, got {residual.dtype}")
        ld_r, r_at = _matrix("residual", residual, index, rows, cols)[2], residual.data_ptr()
    if counter is not None:
        _need(counter.dtype == torch.int64 and counter.numel() == 1 and counter.get_device() == index,
              "counter must be one int64 value on the device")
        counter_at = counter.data_ptr()
    _call(index, "muon_dropout", _dropout_args(
        x.data_ptr(), r_at, y.data_ptr(), counter_at, rows, cols, ld, ld_r, ld_y, seed & _U64, offset & _U64,
        p, _dtype(name, x)))
    return y


def dropout(x: torch.Tensor, p: float, seed: int, offset: int = 0, *,
            counter: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x with a share p of its elements zero and the others divided by 1 - p
    (+ residual), rows x cols, fp32 or bf16.

    Which elements are dropped follows from seed, offset and an element's place
    alone, so that no mask is kept: :func:`dropout_backward` is given the same
    two.  Calls of one seed need offsets of their own.  p is taken to the
    nearest 2^-16.  counter: one int64 value on the device that is added to the
    offset when the kernel runs (captured graphs).  out may be x or residual, and
    otherwise shares no memory with them."""
    return _drop("x", x, p, seed, offset, counter, residual, out)


def dropout_backward(dy: torch.Tensor, p: float, seed: int, offset: int = 0, *,
                     counter: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of dropout's x (that of the residual is dy itself)."""
    return _drop("dy", dy, p, seed, offset, counter, None, out)
