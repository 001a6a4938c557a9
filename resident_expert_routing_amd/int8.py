"""Rows and matrix products in 8-bit integers, with a scale for each token and channel.

    q, scale = quantize(x)                       # activations, or weights [channels, K]
    y = matmul(q, scale, wq, wscale)             # dense
    y = matmul(q, scale, wq, wscale, offsets=buf.slot_offsets, index=buf.perm, index_div=k,
               swiglu=True)                      # experts' gate and up over a bucketing

`Int8Experts` holds the experts of a layer in this format and runs them on
moe_route's bucketing, in place of moe_experts_forward.  All calls run on the
current stream of their tensors' device and synchronise nothing.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from . import binding as B
from .rows import (DTYPES, RowOrder, combine, dtype_of, gpu_tensor, no_tangent, on_its_device,
                   row_major, stream_of)

_lib = B.load()


def _rows16(*shape, device) -> torch.Tensor:
    """An int8 tensor whose rows (last axis) start at multiples of 16 bytes."""
    width = B.moe_int8_row_bytes(shape[-1])
    if width == 0:
        raise ValueError(f"rows of {shape[-1]} elements")
    q = torch.empty(*shape[:-1], width, dtype=torch.int8, device=device)
    return q if width == shape[-1] else q[..., :shape[-1]]


def pad_rows(q: torch.Tensor) -> torch.Tensor:
    """q [..., K] with its rows laid out as the products read them: contiguous,
    at multiples of 16 bytes, groups apart; q itself where it is laid out so."""
    K = q.shape[-1]
    if _laid_out(q):
        return q
    out = _rows16(*q.shape, device=q.device)
    out.copy_(q)
    return out


def _laid_out(q: torch.Tensor) -> bool:
    *lead, K = q.shape
    width = (K + 15) // 16 * 16
    if q.data_ptr() % 16 or (K > 1 and q.stride(-1) != 1):
        return False
    need = width
    for n, s in zip(reversed(lead), reversed(q.stride()[:-1])):
        if n > 1 and (s % 16 or s < need):
            return False
        need = need if n <= 1 else (n - 1) * s + need
    # the padding of the last row has to be inside the memory too
    return q.storage_offset() + need <= q.untyped_storage().nbytes()


def _no_gradient(call: str, *tensors) -> None:
    if forward_ad._current_level >= 0:
        no_tangent(call, *tensors)
    for t in tensors:
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{call} has no gradient: detach its tensors, or call it under "
                             "torch.no_grad()")


def _written(*tensors) -> None:
    """Counts a kernel's write to tensors of the caller's as a change, so that a
    backward pass that kept what they held before is refused."""
    torch.autograd.graph.increment_version([t for t in tensors if not t.is_inference()])


def quantize(x: torch.Tensor, out: tuple[torch.Tensor, torch.Tensor] | None = None):
    """x [M, K] (bf16, fp16 or fp32) -> (q int8 [M, K], scale float32 [M]) with
    x ~= q * scale[:, None]; the scale is the row's largest magnitude over 127.
    `out`: a pair that an earlier call of the same shape returned, to be filled, or
    views of that layout; from K up to the next multiple of 16 a row of q is set
    to zero.
    There is no gradient: tensors that want one, or carry a tangent, are refused."""
    gpu_tensor(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must have shape [M, K], not {list(x.shape)}")
    _no_gradient("quantize", x, *(out or ()))
    dt = dtype_of(x, "x")
    M, K = x.shape
    if max(M, K) > B.MOE_INT_MAX:
        raise B.MoeError(B.MOE_EUNSUPPORTED, "moe_int8_quantize")
    x, stride = row_major(x)
    given = out is not None
    if not given:
        q = _rows16(M, K, device=x.device)
        scale = torch.empty(M, dtype=torch.float32, device=x.device)
    else:
        q, scale = out
        gpu_tensor(q, "q", x.get_device()), gpu_tensor(scale, "scale", x.get_device())
        if q.dtype != torch.int8 or q.shape != x.shape or not _laid_out(q):
            raise ValueError("q must be int8 [M, K] with rows at multiples of 16 bytes")
        if scale.dtype != torch.float32 or scale.numel() != M or not scale.is_contiguous():
            raise ValueError("scale must hold M contiguous float32 values")
    _quantize(x, M, K, stride, dt, q.data_ptr(), _stride(q, 0), scale.data_ptr())
    if given:
        _written(q, scale)
    return q, scale


@on_its_device
def _quantize(x, *args):
    st = _lib.moe_int8_quantize(x.data_ptr(), *args, stream_of(x))
    if st != B.MOE_OK:
        raise B.MoeError(st, "moe_int8_quantize")


def _pointer(t, what: str, dtype: torch.dtype, device: int):
    """The address of a tensor of that type on that GPU; None for None."""
    if t is None:
        return None
    if gpu_tensor(t, what, device).dtype != dtype:
        raise ValueError(f"{what} must be {dtype}")
    return t.data_ptr()


def _stride(q: torch.Tensor, axis: int) -> int:
    """Bytes along `axis` of a laid out tensor (an axis of one has no stride of its own)."""
    if q.shape[axis] > 1:
        return q.stride(axis)
    K = (q.shape[-1] + 15) // 16 * 16
    return K if axis % q.dim() == q.dim() - 2 else q.shape[-2] * _stride(q, -2)


def matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor, *,
           offsets: torch.Tensor | None = None, index: torch.Tensor | None = None,
           index_div: int = 1, swiglu: bool = False, out: torch.Tensor | None = None,
           out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """moe_int8_matmul: out[p, n] = a_scale[r] * b_scale[g, n] * sum_i a[r, i] * b[g, n, i].

    a int8 [rows, K], a_scale float32 [rows]; b int8 [N, K] and b_scale [N], or
    with `offsets` (int32 [G+1]) b [G, N, K] and b_scale [G, N]: rows
    offsets[g] .. offsets[g+1] of out belong to group g.  swiglu: b holds 2N
    rows, gate then up, and out = silu(gate) * up.  `index` (int32 [M]) with
    index_div names the rows of a: r = index[p] // index_div; without it r = p.
    Rows of `out` in no group, or whose index is negative, are left as they
    were (a new `out` starts undefined there); `out` must not overlap an input.
    b has to be laid out with its rows at multiples of 16 bytes (quantize and
    pad_rows do); a is copied if it is not.  There is no gradient: scales and an
    `out` that want one, or carry a tangent, are refused.
    """
    dev = gpu_tensor(a, "a").get_device()
    if a.dtype != torch.int8 or a.dim() != 2:
        raise ValueError("a must be int8 [rows, K]")
    b_at = _pointer(b, "b", torch.int8, dev)
    bs_at = _pointer(b_scale, "b_scale", torch.float32, dev)
    a_rows, K = a.shape
    G = 0 if offsets is None else offsets.numel() - 1
    if b.dim() != (3 if offsets is not None else 2) or b.shape[-1] != K or \
            (offsets is not None and (b.shape[0] != G or G < 1)):
        raise ValueError(f"b {list(b.shape)} does not fit K = {K} and {G} groups")
    wide = b.shape[-2]
    N = wide // 2 if swiglu else wide
    if swiglu and wide % 2:
        raise ValueError("swiglu needs an even number of rows of b")
    if max(a_rows, K, wide, G) > B.MOE_INT_MAX or \
            (index is not None and not B.fits(index_div, index.numel())):
        raise B.MoeError(B.MOE_EUNSUPPORTED, "moe_int8_matmul")
    if a_scale.numel() != a_rows or b_scale.shape != b.shape[:-1]:
        raise ValueError("a_scale and b_scale must have one value for each row of a and b")
    if wide > 1 and b_scale.stride(-1) != 1:
        raise ValueError("the scales of a group must be contiguous")
    if not _laid_out(b):
        raise ValueError("b's rows must start at multiples of 16 bytes: lay it out with pad_rows")
    _no_gradient("matmul", a_scale, b_scale, *(() if out is None else [out]))
    a, a_scale = pad_rows(a), a_scale.contiguous()
    M = a_rows
    if index is not None:
        index, M = index.contiguous(), index.numel()
    if offsets is not None:
        offsets = offsets.contiguous()
    given = out is not None
    if not given:
        if out_dtype not in DTYPES:
            raise ValueError(f"out_dtype must be bfloat16, float16 or float32, not {out_dtype}")
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    elif gpu_tensor(out, "out", dev).shape != (M, N):
        raise ValueError(f"out must have shape [{M}, {N}]")
    od = dtype_of(out, "out")
    if (N > 1 and out.stride(1) != 1) or (M > 1 and out.stride(0) < N):
        raise ValueError("the rows of out must be contiguous and apart")
    _matmul(a, B.Int8MatmulArgs(
        M, N, K, G, 1 if swiglu else 0, a_rows, a.data_ptr(), _stride(a, 0),
        _pointer(a_scale, "a_scale", torch.float32, dev),
        _pointer(index, "index", torch.int32, dev), int(index_div),
        _pointer(offsets, "offsets", torch.int32, dev), b_at, _stride(b, -2),
        _stride(b, 0) if G else 0, bs_at, (b_scale.stride(0) if G > 1 else wide) if G else 0,
        out.data_ptr(), out.stride(0) if M > 1 else N, od))
    if given:
        _written(out)
    return out


@on_its_device
def _matmul(a, args):
    st = _lib.moe_int8_matmul(args, stream_of(a))
    if st != B.MOE_OK:
        raise B.MoeError(st, "moe_int8_matmul")


class Int8Experts:
    """SwiGLU experts of a layer in 8-bit integers, one group for each slot:
    gate_up int8 [S, 2I, H] with scales [S, 2I], down int8 [S, H, I] with scales
    [S, H].  from_weights quantises floating weights slot by slot."""

    def __init__(self, gate_up, gate_up_scale, down, down_scale):
        self.gate_up, self.gate_up_scale = pad_rows(gate_up), gate_up_scale
        self.down, self.down_scale = pad_rows(down), down_scale
        S, two_i, H = gate_up.shape
        if tuple(down.shape) != (S, H, two_i // 2):
            raise ValueError(f"down {list(down.shape)} does not fit gate_up {list(gate_up.shape)}")
        self.S, self.I, self.H = S, two_i // 2, H

    @classmethod
    def empty(cls, S: int, H: int, I: int, device) -> "Int8Experts":
        f32 = dict(dtype=torch.float32, device=device)
        return cls(_rows16(S, 2 * I, H, device=device), torch.empty(S, 2 * I, **f32),
                   _rows16(S, H, I, device=device), torch.empty(S, H, **f32))

    @classmethod
    def from_weights(cls, gate, up, down) -> "Int8Experts":
        """gate, up [S, I, H] and down [S, H, I] in bf16, fp16 or fp32."""
        S, I, H = gate.shape
        e = cls.empty(S, H, I, gate.device)
        for s in range(S):
            e.load(s, gate[s], up[s], down[s])
        return e

    def load(self, slot: int, gate, up, down) -> None:
        """Quantises one expert's floating weights into a slot."""
        I = self.I
        gu, gs = self.gate_up[slot], self.gate_up_scale[slot]
        quantize(gate, (gu[:I], gs[:I]))
        quantize(up, (gu[I:], gs[I:]))
        quantize(down, (self.down[slot], self.down_scale[slot]))

    def check(self, x, T: int, *dtypes) -> None:
        """Refuses token rows that are not [T, H] of a type that quantize takes, on
        the experts' device, or that want a gradient; and other result types."""
        gpu_tensor(x, "x", self.gate_up.get_device())
        dtype_of(x, "x")
        if tuple(x.shape) != (T, self.H):
            raise ValueError(f"x must have shape [{T}, {self.H}], not {list(x.shape)}")
        for d in dtypes:
            if d not in DTYPES:
                raise ValueError(f"rows are bfloat16, float16 or float32, not {d}")
        _no_gradient("Int8Experts", x)

    def rows(self, x, slot_offsets, perm, k: int, out_dtype=torch.float32,
             inner_dtype=torch.bfloat16) -> torch.Tensor:
        """The experts on the rows of a bucketing: token rows x [T, H] ->
        [T*k, H] (as many rows as perm has), row p from token perm[p] // k; rows
        that are in no slot are undefined.  The second products' inputs are
        rounded to inner_dtype before they are quantised: bf16, half the bytes of
        float32 and off by at most 2^-9 of a value where the 8-bit step is 2^-7 of
        the row's largest, whatever x's type; float32 leaves the one rounding to 8
        bits (fp16 overflows at 65504)."""
        self.check(x, x.shape[0], out_dtype, inner_dtype)
        if perm.numel() > x.shape[0] * k:
            raise ValueError(f"perm holds {perm.numel()} values, more than the T*k = "
                             f"{x.shape[0] * k} assignments of x")
        q, s = quantize(x)
        h = matmul(q, s, self.gate_up, self.gate_up_scale, offsets=slot_offsets, index=perm,
                   index_div=k, swiglu=True, out_dtype=inner_dtype)
        hq, hs = quantize(h)
        return matmul(hq, hs, self.down, self.down_scale, offsets=slot_offsets,
                      out_dtype=out_dtype)

    def forward(self, x, slot_offsets, perm, sel_weight, pos=None, *, row_dtype=None,
                inner_dtype=torch.bfloat16) -> torch.Tensor:
        """x [T, H] -> [T, H] in x's type: the layer's experts and their weighted
        sum, from what moe_route wrote for the batch.  The experts' rows are
        rounded to row_dtype (x's type if None: the sum of bf16 rows reads half
        the bytes) before they are weighted and summed; of float32 rows only the
        sum is rounded.  inner_dtype as in rows."""
        T, k = sel_weight.shape
        self.check(x, T)
        order = RowOrder(perm, T, k, pos)
        rows = self.rows(x, slot_offsets, perm, k, row_dtype or x.dtype, inner_dtype)
        return combine(rows, order, sel_weight).to(x.dtype)
