"""Products of ragged groups of rows, one matrix for each group, as a differentiable function.

    order = rows.RowOrder(buf.perm, T, k)                     # after runtime.route(buf, ...)
    h = matmul(x, gate_up, buf.slot_offsets, order=order, swiglu=True)      # [T*k, I]
    y = matmul(h, down, buf.slot_offsets)                                   # [T*k, H]
    out = rows.combine(y, order, buf.sel_weight)

`GroupedExperts` does these for a layer.  Rows and matrices are of one type (bf16, fp16 or
fp32; sums are float32), and gradients go to both (moe_grouped_matmul, moe_grouped_outer,
moe_swiglu_backward).  A call that is recorded keeps copies of the offsets and of the
order, which the next moe_route may write over, and with SwiGLU the products before it in
float32; rows are kept as they are for the matrices' gradient, matrices for the rows'.
There is no forward-mode derivative: tensors that carry a tangent are refused.  Calls run
on the current stream of their tensors' device and synchronise nothing.  A gradient
captured into a graph is taken with torch.autograd.grad, or with no graph made outside the
capture alive over the same leaves: torch ties a leaf's accumulation to the stream that
first used it.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from . import binding as B
from .rows import (RowOrder, _gather, combine, dtype_of, gpu_tensor, no_tangent, on_its_device,
                   row_major, stream_of)

_lib = B.load()
_MOST = 1 << 24  # contraction of a product; the gradients' products have b's rows there


def _matrices(b: torch.Tensor):
    """(b, whether its inputs lie across its rows, elements from row to row and from group
    to group) of matrices [G, N, K]; a copy of them where neither N nor K is contiguous."""
    G, n, k = b.shape
    group, down, right = b.stride()
    if (k == 1 or right == 1) and (n == 1 or down >= k):
        return b, False, (down if n > 1 else k), (group if G > 1 else 0)
    if (n == 1 or down == 1) and (k == 1 or right >= n):
        return b, True, (right if k > 1 else n), (group if G > 1 else 0)
    return b.contiguous(), False, k, n * k


@on_its_device
def _products(a, b, offsets, index, index_div, M, N, swiglu, out, zero, keep, pos=None):
    """out [M, N], and with `keep` the products before SwiGLU; b as _matrices has it."""
    b, across, down, group = b
    a, stride = row_major(a)
    K, G = a.shape[1], offsets.numel() - 1
    pre = torch.empty((M, 2 * N), dtype=torch.float32, device=a.device) if keep else None
    st = _lib.moe_grouped_matmul(B.GroupedMatmulArgs(
        M, N, K, G, dtype_of(a, "a"), swiglu, across, zero, a.shape[0], a.data_ptr(), stride,
        None if index is None else index.data_ptr(), index_div, offsets.data_ptr(), b.data_ptr(),
        down, group, out.data_ptr(), out.stride(0) if M > 1 else N,
        None if pre is None else pre.data_ptr(), 2 * N, dtype_of(out, "out"),
        None if pos is None else pos.data_ptr()), stream_of(a))
    if st != B.MOE_OK:
        raise B.MoeError(st, "moe_grouped_matmul")
    return pre


@on_its_device
def _outer(left, left_index, left_div, right, right_index, right_div, offsets, M, pos=None):
    """[G, L, R]: the sums of left[p] x right[p] over each group's rows."""
    left, ls = row_major(left)
    right, rs = row_major(right)
    L, R, G = left.shape[1], right.shape[1], offsets.numel() - 1
    out = torch.empty((G, L, R), dtype=left.dtype, device=left.device)
    at = lambda t: None if t is None else t.data_ptr()
    dt = dtype_of(left, "left")
    need = _lib.moe_grouped_outer_ws_bytes(M, L, R, G, dt)
    ws = torch.empty(need, dtype=torch.uint8, device=left.device) if need else None
    st = _lib.moe_grouped_outer(B.GroupedOuterArgs(
        M, L, R, G, dt, left.shape[0], right.shape[0], left.data_ptr(), ls,
        at(left_index), left_div, right.data_ptr(), rs, at(right_index), right_div,
        offsets.data_ptr(), out.data_ptr(), R, L * R, at(ws), need, at(pos)), stream_of(left))
    if st != B.MOE_OK:
        raise B.MoeError(st, "moe_grouped_outer")
    return out


@on_its_device
def _swiglu_backward(dout, pre):
    dout, stride = row_major(dout)
    M, N = dout.shape
    dpre = torch.empty((M, 2 * N), dtype=dout.dtype, device=dout.device)
    st = _lib.moe_swiglu_backward(M, N, dtype_of(dout, "the gradient"), pre.data_ptr(), 2 * N,
                                  dout.data_ptr(), stride, dpre.data_ptr(), 2 * N,
                                  stream_of(pre))
    if st != B.MOE_OK:
        raise B.MoeError(st, "moe_swiglu_backward")
    return dpre


class _Matmul(torch.autograd.Function):
    @staticmethod
    def forward(ctx, a, b, offsets, order, index, index_div, M, N, swiglu):
        out = torch.empty((M, N), dtype=a.dtype, device=a.device)
        keep = order.kept() if order is not None else None
        idx, pos = (keep.perm, keep.pos) if keep is not None else (index, None)
        taken = _matrices(b)
        pre = _products(a, taken, offsets, idx, index_div, M, N, swiglu, out, True, swiglu, pos)
        # each gradient reads the other operand, and b's the rows' names
        da, db = ctx.needs_input_grad[:2]
        named = None if not db else keep.perm if keep is not None else \
            index.clone() if index is not None else None
        ctx.save_for_backward(a if db else None, b if da else None, offsets.clone(), named, pos, pre)
        ctx.sizes = M, N, a.shape[1], swiglu, index_div, taken[1]
        ctx.tokens = (order.T, order.k) if order is not None else None
        return out

    @staticmethod
    def backward(ctx, grad):
        if torch.is_grad_enabled():
            raise RuntimeError("grouped products have no second derivative: take their gradient "
                               "without create_graph")
        no_tangent("the gradient of grouped products", grad)
        a, b, offsets, named, pos, pre = ctx.saved_tensors
        M, N, K, swiglu, div, across = ctx.sizes
        dz = _swiglu_backward(grad, pre) if swiglu else grad
        da = db = None
        if ctx.needs_input_grad[0]:
            b, across, down, group = _matrices(b)
            # a token's rows are summed before they are rounded
            rows = torch.float32 if ctx.tokens is not None else grad.dtype
            da = torch.empty((M, K), dtype=rows, device=grad.device)
            _products(dz, (b, not across, down, group), offsets, None, 1, M, K, False, da, True,
                      False)
            if ctx.tokens is not None:
                da = _gather(da, RowOrder.of(None, pos, *ctx.tokens), None)[0].to(grad.dtype)
        if ctx.needs_input_grad[1]:
            if across:
                db = _outer(a, named, div, dz, None, 1, offsets, M, pos).transpose(1, 2)
            else:
                db = _outer(dz, None, 1, a, named, div, offsets, M, pos)
        return da, db, None, None, None, None, None, None, None


def matmul(a: torch.Tensor, b: torch.Tensor, offsets: torch.Tensor, *,
           order: RowOrder | None = None, index: torch.Tensor | None = None, index_div: int = 1,
           swiglu: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """moe_grouped_matmul: out[p, n] = sum_i a[r, i] * b[g, n, i] for the rows p of group g,
    offsets[g] <= p < offsets[g+1] (offsets int32 [G+1], ascending).

    a [rows, K] and b [G, N, K] in one type; b's matrices may be contiguous along either
    axis (a transposed view of [G, K, N] is taken as it lies; other layouts are copied).
    swiglu: b holds 2N rows, gate then up, and out = silu(gate) * up.  The rows of a: r = p;
    with `order` (rows.RowOrder of T*k assignments) the token row perm[p] // k, and a has
    T rows (the earlier row of an assignment that it names twice has none, as in
    rows.dispatch); with `index` (int32 [M]) r = index[p] // index_div.  Gradients go to a and b;
    that of rows named by `index` has to be taken with `order`, which knows each token's
    rows.  Rows of out that nothing is computed for (in no group, or whose index is
    negative) are zero; in an `out` of the caller's, [M, N] with contiguous rows, which is
    for calls that record no gradient and must not overlap an input, they are left as they
    were."""
    dev = gpu_tensor(a, "a").get_device()
    gpu_tensor(b, "b", dev)
    dt = dtype_of(a, "a")
    if b.dtype != a.dtype:
        raise ValueError(f"a is {a.dtype}, b {b.dtype}")
    if gpu_tensor(offsets, "offsets", dev).dtype != torch.int32 or offsets.dim() != 1 or \
            offsets.numel() < 2:
        raise ValueError("offsets must be int32 [G+1]")
    G = offsets.numel() - 1
    if a.dim() != 2 or b.dim() != 3 or b.shape[0] != G or b.shape[2] != a.shape[1]:
        raise ValueError(f"a {list(a.shape)}, b {list(b.shape)} and {G} groups do not fit")
    rows, K = a.shape
    wide = b.shape[1]
    if K < 1 or wide < 1 or (swiglu and wide % 2):
        raise ValueError(f"b {list(b.shape)}: swiglu needs an even number of rows, and K and N "
                         "are at least 1")
    N = wide // 2 if swiglu else wide
    M, own_index, pos = rows, None, None
    if order is not None:
        if index is not None:
            raise ValueError("order or index, not both")
        if order.device != dev or rows != order.T:
            raise ValueError(f"a must hold the order's {order.T} token rows, on its device")
        M, own_index, pos, index_div = order.T * order.k, order.perm, order.pos, order.k
    elif index is not None:
        if gpu_tensor(index, "index", dev).dtype != torch.int32:
            raise ValueError("index must be int32")
        index = own_index = index.contiguous()
        M = index.numel()
    if max(rows, K, wide, G, M) > B.MOE_INT_MAX or not B.fits(index_div):
        raise B.MoeError(B.MOE_EUNSUPPORTED, "moe_grouped_matmul")
    if forward_ad._current_level >= 0:
        no_tangent("grouped.matmul", a, b, out)
    offsets = offsets.contiguous()
    if torch.is_grad_enabled() and (a.requires_grad or b.requires_grad or
                                    (out is not None and out.requires_grad)):
        if out is not None:
            raise ValueError("a call with `out` has no gradient: detach its tensors, or call it "
                             "under torch.no_grad()")
        if a.requires_grad and index is not None:
            raise ValueError("the gradient of rows named by index needs `order`")
        if wide > _MOST or (a.requires_grad and order is not None and order.k > B.MOE_MAX_K):
            raise B.MoeError(B.MOE_EUNSUPPORTED, "the gradient of grouped products")
        return _Matmul.apply(a, b, offsets, order, index, int(index_div), M, N, bool(swiglu))
    given = out is not None
    if not given:
        out = torch.empty((M, N), dtype=a.dtype, device=a.device)
    else:
        if gpu_tensor(out, "out", dev).shape != (M, N) or dtype_of(out, "out") != dt:
            raise ValueError(f"out must be {a.dtype} [{M}, {N}]")
        if (N > 1 and out.stride(1) != 1) or (M > 1 and out.stride(0) < N):
            raise ValueError("the rows of out must be contiguous and apart")
    _products(a, _matrices(b), offsets, own_index, int(index_div), M, N, bool(swiglu), out,
              not given, False, pos)
    if given and not out.is_inference():
        torch.autograd.graph.increment_version([out])
    return out


class GroupedExperts:
    """SwiGLU experts of a layer in floating point, one group for each slot: gate_up
    [S, 2I, H] (gate rows, then up rows) and down [S, H, I], any layout that matmul takes.
    Both may be parameters of a model: forward passes gradients to them, to the token rows
    and to the weights of the sum."""

    def __init__(self, gate_up: torch.Tensor, down: torch.Tensor):
        if gate_up.dim() != 3 or gate_up.shape[1] % 2 or tuple(down.shape) != \
                (gate_up.shape[0], gate_up.shape[2], gate_up.shape[1] // 2):
            raise ValueError(f"down {list(down.shape)} does not fit gate_up {list(gate_up.shape)}")
        self.gate_up, self.down = gate_up, down
        self.S, self.I, self.H = down.shape[0], down.shape[2], down.shape[1]
        self._check_matrices()

    def _check_matrices(self) -> None:
        gate_up, down = self.gate_up, self.down
        dtype_of(gate_up, "gate_up")
        if down.dtype != gate_up.dtype or down.device != gate_up.device:
            raise ValueError(f"gate_up is {gate_up.dtype} on {gate_up.device}, down {down.dtype} on "
                             f"{down.device}")

    def check(self, x, T: int) -> None:
        """Refuses token rows that are not [T, H] of the experts' type and device, matrices
        that are not on a GPU or differ in either (a model's parameters may be moved or cast
        after they were given), and tangents."""
        self._check_matrices()
        gpu_tensor(self.gate_up, "gate_up")
        if forward_ad._current_level >= 0:
            no_tangent("GroupedExperts", x, self.gate_up, self.down)
        gpu_tensor(x, "x", self.gate_up.get_device())
        if x.dtype != self.gate_up.dtype or tuple(x.shape) != (T, self.H):
            raise ValueError(f"x must be {self.gate_up.dtype} [{T}, {self.H}], not {x.dtype} "
                             f"{list(x.shape)}")

    def forward(self, x, slot_offsets, perm, sel_weight, pos=None) -> torch.Tensor:
        """x [T, H] -> [T, H]: the layer's experts and their weighted sum, from what
        moe_route wrote for the batch.  The rows between the products and before the sum
        are rounded to x's type, as the next product's operand has to be and as half the bytes
        of float32 rows: off by at most half a step each, 2^-8 of a value in bf16."""
        T, k = sel_weight.shape
        self.check(x, T)
        order = RowOrder(perm, T, k, pos)
        h = matmul(x, self.gate_up, slot_offsets, order=order, swiglu=True)
        return combine(matmul(h, self.down, slot_offsets), order, sel_weight)
