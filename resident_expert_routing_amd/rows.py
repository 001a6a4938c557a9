"""Token rows in the order of the slots and back, as differentiable torch functions.

    order = RowOrder(buf.perm, T, k)            # perm as moe_route wrote it
    rows = dispatch(x, order)                   # [T*k, H], row p: token perm[p] // k
    ... any experts, slot s on rows slot_offsets[s] .. slot_offsets[s+1] ...
    out = combine(rows, order, buf.sel_weight)  # [T, H]

Both take bf16, fp16 or fp32 rows and float32 weights, and pass gradients to the
rows and to the weights (moe_dispatch_backward, moe_combine_backward).  A call
that is recorded keeps copies of the order and of the weights, since the next
moe_route may write over both before the backward pass; rows that the weights'
gradient needs are kept as they are.  There is no forward-mode derivative: tensors
that carry a tangent are refused.  Calls run on the current stream of the
rows' device and synchronise nothing.  A gradient captured into a graph is taken
with torch.autograd.grad, or with no graph made outside the capture alive over
the same leaves: torch ties a leaf's accumulation to the stream that first used it.
"""
from __future__ import annotations

import functools

import torch
from torch.autograd import forward_ad

from . import binding as B

_lib = B.load()

DTYPES = {torch.bfloat16: B.MOE_DT_BF16, torch.float16: B.MOE_DT_FP16,
          torch.float32: B.MOE_DT_FP32}


def stream_of(t: torch.Tensor) -> int:
    """The handle of the current stream of the tensor's device."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def on_its_device(call):
    """`call`, with the device of its first argument (a tensor) the current one."""
    @functools.wraps(call)
    def run(t, *args):
        if t.get_device() == torch.cuda.current_device():
            return call(t, *args)
        with torch.cuda.device(t.device):
            return call(t, *args)
    return run


def dtype_of(t: torch.Tensor, what: str) -> int:
    code = DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be bfloat16, float16 or float32, not {t.dtype}")
    return code


def gpu_tensor(t, what: str, device: int | None = None) -> torch.Tensor:
    """t, a tensor on a GPU (on GPU `device`, where that is given)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a tensor on a GPU")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{what} is on {t.device}, other tensors on GPU {device}")
    return t


def no_tangent(call: str, *tensors) -> None:
    """Refuses tensors that carry a forward-mode tangent (None among them is none):
    the kernels see a tensor's values only, and a result without a tangent would
    pass for one of derivative zero.  Outside every dual_level no tensor has one;
    small calls look at forward_ad._current_level themselves, without this call."""
    if forward_ad._current_level < 0:
        return
    for t in tensors:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError(f"{call} has no forward-mode derivative: a tensor carries a tangent")


def row_major(t: torch.Tensor) -> tuple[torch.Tensor, int]:
    """(t, elements from row to row) of a matrix whose rows are contiguous and
    apart; other layouts (transposed, expanded) are copied first."""
    n, width = t.shape
    down, across = t.stride()
    if (across == 1 or width == 1) and (n <= 1 or down >= width):
        return t, down if n > 1 else width
    return t.contiguous(), width


@on_its_device
def _positions(perm, T, k):
    both = torch.empty((2, T, k), dtype=torch.int32, device=perm.device)
    pos, copy = both.unbind()
    B.check(B.moe_positions(perm, T, k, pos, copy, stream_of(perm)), "moe_positions")
    return pos, copy


class RowOrder:
    """The order of a batch's T*k assignments by slot: perm (row -> assignment,
    int32, as moe_route wrote it, -1 behind the last row that is used) and its
    inverse pos [T, k] (assignment -> row, -1 for none).  moe_positions computes
    pos and copies perm, so a later moe_route may write over the caller's; a pos
    that the caller already has is taken as it is, with perm, and both are
    copied when a dispatch or combine is recorded for its backward pass; it has to
    be the inverse of this perm.  An order used on another stream than the one it
    was made on is kept until that stream is done with it, or announced to the
    allocator as other tensors are (order.pos.record_stream(stream); of an order
    with a pos of the caller's, order.perm too)."""

    def __init__(self, perm: torch.Tensor, T: int, k: int, pos: torch.Tensor | None = None):
        self.T, self.k = int(T), int(k)
        n = self.T * self.k
        if self.T < 0 or self.k < 1 or n > B.MOE_INT_MAX:
            raise ValueError(f"{T} tokens of {k} picks: at most 2^31 - 1 assignments, k of 1 "
                             f"to {B.MOE_MAX_K}")
        if gpu_tensor(perm, "perm").dtype != torch.int32 or perm.numel() != n:
            raise ValueError(f"perm must hold T*k = {n} int32 values")
        self.device = perm.get_device()
        self.own = pos is None
        if self.own:
            self.pos, self.perm = _positions(perm.contiguous(), self.T, self.k)
            return
        if gpu_tensor(pos, "pos", self.device).dtype != torch.int32 or \
                pos.shape not in ((self.T, self.k), (n,)):
            raise ValueError(f"pos must be int32 [{self.T}, {self.k}]")
        self.pos, self.perm = pos.contiguous(), perm.contiguous()

    def kept(self) -> "RowOrder":
        """The order in tensors of its own."""
        if self.own:
            return self
        order = object.__new__(RowOrder)
        order.T, order.k, order.device, order.own = self.T, self.k, self.device, True
        both = torch.cat((self.pos.view(-1), self.perm.view(-1)))
        order.pos, order.perm = both.view(2, self.T, self.k).unbind()
        return order


def _weights(weight, order: RowOrder):
    if weight is None:
        return None
    gpu_tensor(weight, "weight", order.device)
    if weight.dtype != torch.float32 or \
            weight.shape not in ((order.T, order.k), (order.T * order.k,)):
        raise ValueError(f"weight must be float32 [{order.T}, {order.k}]")
    return weight.contiguous()


# The two moves.  Small batches are bound by what happens here on the host, so
# the C entries are called with plain numbers.
def _move_rows(entry, what, n, src, order, weight, perm, other=None):
    """entry(src) -> rows or token rows [n, H]; with `other` (the forward input)
    the weights' gradient too."""
    if order.device != torch.cuda.current_device():
        with torch.cuda.device(order.device):
            return _move_rows(entry, what, n, src, order, weight, perm, other)
    dt = dtype_of(src, "rows")
    H, T, k = src.shape[1], order.T, order.k
    if H > B.MOE_INT_MAX:
        raise B.MoeError(B.MOE_EUNSUPPORTED, what)
    src, stride = row_major(src)
    dst = torch.empty((n, H), dtype=src.dtype, device=src.device)
    dw, dwp, op, ostride = None, None, None, 0
    if other is not None:
        other, ostride = row_major(other)
        dw = torch.empty((T, k), dtype=torch.float32, device=src.device)
        dwp, op = dw.data_ptr(), other.data_ptr()
    st = entry(B.RowsArgs(T, H, k, dt, None if perm is None else perm.data_ptr(),
                          order.pos.data_ptr(), None if weight is None else weight.data_ptr(),
                          src.data_ptr(), stride, dst.data_ptr(), H, op, ostride, dwp),
               torch._C._cuda_getCurrentRawStream(order.device))
    if st != B.MOE_OK:
        raise B.MoeError(st, what)
    return dst, dw


def _spread(src, order, weight, rows=None):
    """Token rows to rows; with `rows` (the forward rows) the weights' gradient too."""
    if rows is None:
        return _move_rows(_lib.moe_dispatch, "moe_dispatch", order.T * order.k, src, order, weight,
                          order.perm)
    return _move_rows(_lib.moe_combine_backward, "moe_combine_backward", order.T * order.k, src,
                      order, weight, order.perm, rows)


def _gather(src, order, weight, tokens=None):
    """Rows to token rows; with `tokens` (the forward token rows) the weights' gradient too."""
    if tokens is None:
        return _move_rows(_lib.moe_combine, "moe_combine", order.T, src, order, weight, None)
    return _move_rows(_lib.moe_dispatch_backward, "moe_dispatch_backward", order.T, src, order,
                      weight, None, tokens)


class _Move(torch.autograd.Function):
    """forward: `there`; backward: `back`, the other of _spread and _gather."""

    @staticmethod
    def forward(ctx, src, weight, order, there, back):
        w = _weights(weight, order)
        ctx.order, ctx.back = order.kept(), back
        wants = weight is not None and ctx.needs_input_grad[1]
        kept = w.clone() if w is not None and w.data_ptr() == weight.data_ptr() else w
        ctx.save_for_backward(src if wants else None, kept)
        ctx.wshape = weight.shape if wants else None
        return there(src, order, w)[0]

    @staticmethod
    def backward(ctx, grad):
        if torch.is_grad_enabled():
            raise RuntimeError("dispatch and combine have no second derivative: take their "
                               "gradient without create_graph")
        no_tangent("the gradient of dispatch and combine", grad)
        src, w = ctx.saved_tensors
        dsrc, dw = ctx.back(grad, ctx.order, w, src)
        if dw is not None:
            dw = dw.view(ctx.wshape)
        return dsrc, dw, None, None, None


def _move(src, weight, order, there, back):
    if forward_ad._current_level >= 0:
        no_tangent("a call of dispatch or combine", src, weight)
    if torch.is_grad_enabled() and (src.requires_grad
                                    or (weight is not None and weight.requires_grad)):
        return _Move.apply(src, weight, order, there, back)
    return there(src, order, _weights(weight, order))[0]


def _check(src: torch.Tensor, n: int, order: RowOrder, what: str) -> None:
    gpu_tensor(src, what, order.device)
    if src.dim() != 2 or src.shape[0] != n:
        raise ValueError(f"{what} must have shape [{n}, H], not {list(src.shape)}")


def dispatch(x: torch.Tensor, order: RowOrder, weight: torch.Tensor | None = None) -> torch.Tensor:
    """x [T, H] -> rows [T*k, H]: row p is x[perm[p] // k], times its weight if
    `weight` [T, k] is given; rows that perm does not use are zero, and so is the
    earlier row of an assignment that perm names twice."""
    _check(x, order.T, order, "x")
    return _move(x, weight, order, _spread, _gather)


def combine(rows: torch.Tensor, order: RowOrder,
            weight: torch.Tensor | None = None) -> torch.Tensor:
    """rows [T*k, H] -> out [T, H]: each token's rows, weighted and summed in
    float32 over ascending picks; a token without rows gets zeros."""
    _check(rows, order.T * order.k, order, "rows")
    return _move(rows, weight, order, _gather, _spread)
