"""Products with 4-bit weights and a scale for each group of weights.

    w = quantize(weight, group=128)              # [N, K] or [G, N, K] in bf16, fp16 or fp32
    w = pack(codes, scale, zero)                 # codes 0..15 that another program quantised
    y = matmul(x, w)                             # dense
    y = matmul(x, w, offsets=buf.slot_offsets, index=buf.perm, index_div=k, swiglu=True)

`Int4Experts` holds the experts of a layer in this format and runs them on moe_route's
bucketing, in place of moe_experts_forward.  Made for few rows of each group (decode), whose
time is that of reading the weights.  All calls run on the current stream of their tensors'
device and synchronise nothing.  There is no gradient.
"""
from __future__ import annotations

import torch

from . import binding as B
from .int8 import _no_gradient, _written
from .rows import (DTYPES, RowOrder, combine, dtype_of, gpu_tensor, on_its_device, row_major,
                   stream_of)

_lib = B.load()
GROUPS = (32, 64, 128)
SCALES = {torch.bfloat16: B.MOE_DT_BF16, torch.float16: B.MOE_DT_FP16}


def _up(v: int, m: int) -> int:
    return -(-v // m) * m


class Int4Weight:
    """Matrices [N, K], or [G, N, K], in 4 bits, as moe_int4_matmul reads them: weight =
    scale * (code - zero), a scale and zero point for each `group` weights of a row.

    codes  uint8 [.., ceil(N/16), ceil(K/128), 16, 64]: tiles of 16 rows by 128 weights, a
           row's 64 bytes sixteen words of eight consecutive weights, weight 2j of a word at bit
           4j, weight 2j+1 at bit 16+4j
    scale  bf16 or fp16 [.., ceil(N/16), groups of the padded K, 16]
    zero   uint8 like scale, or None: all 8
    The last three axes are contiguous; matrices may lie at any distance (multiples of 16
    bytes, of four scales and four zero points).  Padding may hold anything."""

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor, zero: torch.Tensor | None = None,
                 *, N: int, K: int):
        dev = gpu_tensor(codes, "codes").get_device()
        gpu_tensor(scale, "scale", dev)
        if N < 1 or K < 1 or not B.moe_int4_code_bytes(N, K):
            raise ValueError(f"a matrix of {N} x {K}")
        blocks, chunks = _up(N, 16) // 16, _up(K, 128) // 128
        if codes.dtype != torch.uint8 or codes.dim() not in (4, 5) or \
                tuple(codes.shape[-4:]) != (blocks, chunks, 16, 64):
            raise ValueError(f"codes must be uint8 [.., {blocks}, {chunks}, 16, 64], not "
                             f"{codes.dtype} {list(codes.shape)}")
        if scale.dtype not in SCALES:
            raise ValueError(f"scales are bfloat16 or float16, not {scale.dtype}")
        lead = tuple(codes.shape[:-4])
        groups = scale.shape[-2] if scale.dim() == len(lead) + 3 else 0
        if groups < 1 or tuple(scale.shape[:-2]) != (*lead, blocks) or scale.shape[-1] != 16 or \
                chunks * 128 % groups or chunks * 128 // groups not in GROUPS:
            raise ValueError(f"scale {list(scale.shape)} does not fit groups of 32, 64 or 128 "
                             f"weights of {list(lead)} matrices {N} x {K}")
        if zero is not None and (gpu_tensor(zero, "zero", dev).dtype != torch.uint8
                                 or zero.shape != scale.shape):
            raise ValueError("zero must be uint8 of scale's shape")
        _no_gradient("Int4Weight", scale)
        self.group = chunks * 128 // groups
        self.N, self.K, self.G = int(N), int(K), (lead[0] if lead else 0)
        for t, what, unit, inner in ((codes, "codes", 16, 4), (scale, "scale", 4, 3),
                                     (zero, "zero", 4, 3)):
            if t is None:
                continue
            one = t[0] if lead and lead[0] else t
            if lead and not lead[0]:
                raise ValueError("no matrices")
            if not one.is_contiguous() or t.data_ptr() % (unit * t.element_size()) or \
                    (lead and lead[0] > 1 and t.stride(0) % unit):
                raise ValueError(f"{what}: a matrix must be contiguous, at multiples of "
                                 f"{unit * t.element_size()} bytes")
        self.codes, self.scale, self.zero = codes, scale, zero
        far = lambda t: 0 if t is None or not self.G else t.stride(0) if self.G > 1 else t.numel()
        self._far = far(codes), far(scale), far(zero)

    def _args(self):
        """The matrices' part of moe_int4_matmul's arguments."""
        codes, scale, zero = self.codes, self.scale, self.zero
        return (self.group, codes.data_ptr(), self._far[0], scale.data_ptr(), self._far[1],
                SCALES[scale.dtype], None if zero is None else zero.data_ptr(), self._far[2])

    @property
    def device(self) -> torch.device:
        return self.codes.device

    @classmethod
    def empty(cls, *shape: int, group: int = 128, zeros: bool = False,
              scale_dtype: torch.dtype = torch.bfloat16, device="cuda") -> "Int4Weight":
        """Matrices [N, K] or [G, N, K] whose contents are to be loaded."""
        *lead, N, K = shape
        if group not in GROUPS:
            raise ValueError(f"groups are of 32, 64 or 128 weights, not {group}")
        blocks, chunks = _up(N, 16) // 16, _up(K, 128) // 128
        scale = torch.empty(*lead, blocks, chunks * 128 // group, 16, dtype=scale_dtype,
                            device=device)
        return cls(torch.empty(*lead, blocks, chunks, 16, 64, dtype=torch.uint8, device=device),
                   scale, torch.empty_like(scale, dtype=torch.uint8) if zeros else None, N=N, K=K)

    def __getitem__(self, g: int) -> "Int4Weight":
        """Matrix g of several."""
        if not self.G:
            raise ValueError("one matrix has no others")
        return Int4Weight(self.codes[g], self.scale[g], None if self.zero is None else self.zero[g],
                          N=self.N, K=self.K)

    def load(self, w: torch.Tensor, row: int = 0) -> None:
        """Quantises floating weights w [n, K] into rows row .. row + n of one matrix, both
        multiples of 16 where rows follow (moe_int4_quantize)."""
        if self.G:
            raise ValueError("load fills one matrix: take it by its number first")
        gpu_tensor(w, "w", self.codes.get_device())
        dt = dtype_of(w, "w")
        _no_gradient("Int4Weight.load", w)
        if w.dim() != 2 or w.shape[1] != self.K or row < 0 or row % 16 or \
                row + w.shape[0] > self.N or \
                (w.shape[0] % 16 and row + w.shape[0] != self.N):
            raise ValueError(f"weights {list(w.shape)} at row {row} do not fit {self.N} x "
                             f"{self.K} in sixteens")
        w, stride = row_major(w)
        at = row // 16
        _quantize(w, w.shape[0], self.K, stride, dt, self.group, self.codes[at:].data_ptr(),
                  self.scale[at:].data_ptr(), SCALES[self.scale.dtype],
                  None if self.zero is None else self.zero[at:].data_ptr())
        _written(*(t for t in (self.codes, self.scale, self.zero) if t is not None))

    def dequantize(self, dtype: torch.dtype = torch.float32) -> torch.Tensor:
        """The weights as numbers, [N, K] or [G, N, K] (elementary torch operations)."""
        c = self.codes
        pairs = torch.stack([c & 15, c >> 4], -1).view(*c.shape[:-1], 16, 2, 4)  # word, parity, pair
        c = pairs.transpose(-1, -2).reshape(*c.shape[:-1], 128).transpose(-2, -3)
        c = c.reshape(*c.shape[:-4], self.codes.shape[-4] * 16, -1).float()
        wide = lambda t: t.float().transpose(-1, -2).reshape(*t.shape[:-3], t.shape[-3] * 16, -1) \
            .repeat_interleave(self.group, dim=-1)
        w = (c - (8.0 if self.zero is None else wide(self.zero))) * wide(self.scale)
        return w[..., :self.N, :self.K].to(dtype)


@on_its_device
def _quantize(w, *args):
    st = _lib.moe_int4_quantize(w.data_ptr(), *args, stream_of(w))
    if st != B.MOE_OK:
        raise B.MoeError(st, "moe_int4_quantize")


def quantize(w: torch.Tensor, group: int = 128, *, zeros: bool = False,
             scale_dtype: torch.dtype = torch.bfloat16) -> Int4Weight:
    """Floating weights [N, K] or [G, N, K] as an Int4Weight (moe_int4_quantize): scales of
    max |w| / 7, or with `zeros` of (max - min) / 15 and a zero point for each group."""
    gpu_tensor(w, "w")
    dtype_of(w, "w")
    if w.dim() not in (2, 3):
        raise ValueError(f"weights must be [N, K] or [G, N, K], not {list(w.shape)}")
    if scale_dtype not in SCALES:
        raise ValueError(f"scales are bfloat16 or float16, not {scale_dtype}")
    _no_gradient("int4.quantize", w)
    out = Int4Weight.empty(*w.shape, group=group, zeros=zeros, scale_dtype=scale_dtype,
                           device=w.device)
    for g in range(out.G) if out.G else (None,):
        (out if g is None else out[g]).load(w if g is None else w[g])
    return out


def pack(codes: torch.Tensor, scale: torch.Tensor, zero: torch.Tensor | None = None, *,
         group: int = 128) -> Int4Weight:
    """An Int4Weight of codes 0..15 that exist already: codes uint8 [.., N, K], scale (bf16 or
    fp16) and zero (uint8, or None: 8) [.., N, ceil(K / group)].  For loading: elementary
    torch operations, matrix by matrix.  There is no gradient: scales that want one, or carry
    a tangent, are refused."""
    dev = gpu_tensor(codes, "codes").get_device()
    gpu_tensor(scale, "scale", dev)
    *lead, N, K = codes.shape
    live = -(-K // group) if group in GROUPS else 0
    if codes.dtype != torch.uint8 or codes.dim() not in (2, 3) or \
            tuple(scale.shape) != (*lead, N, live):
        raise ValueError(f"codes {list(codes.shape)}, scale {list(scale.shape)} and groups of "
                         f"{group} do not fit")
    if zero is not None and (gpu_tensor(zero, "zero", dev).shape != scale.shape
                             or zero.dtype != torch.uint8):
        raise ValueError("zero must be uint8 of scale's shape")
    _no_gradient("int4.pack", scale)
    out = Int4Weight.empty(*codes.shape, group=group, zeros=zero is not None,
                           scale_dtype=scale.dtype, device=codes.device)
    for g in range(out.G) if out.G else (None,):
        to, at = (out, ()) if g is None else (out[g], (g,))
        Np, Kp = to.codes.shape[0] * 16, to.codes.shape[1] * 128
        c = torch.zeros(Np, Kp, dtype=torch.uint8, device=codes.device)
        c[:N, :K] = codes[at]
        t = c.view(Np // 16, 16, Kp // 128, 16, 4, 2).permute(0, 2, 1, 3, 5, 4)
        to.codes.copy_((t[..., 0::2] | (t[..., 1::2] << 4)).reshape(to.codes.shape))
        for src, dst in ((scale, to.scale), (zero, to.zero)):
            if src is not None:
                s = torch.zeros(Np, Kp // group, dtype=src.dtype, device=codes.device)
                s[:N, :live] = src[at]
                dst.copy_(s.view(Np // 16, 16, -1).transpose(1, 2))
    return out


def matmul(a: torch.Tensor, w: Int4Weight, *, offsets: torch.Tensor | None = None,
           index: torch.Tensor | None = None, index_div: int = 1, swiglu: bool = False,
           out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """moe_int4_matmul: out[p, n] = sum_i a[r, i] * w[g, n, i].

    a [rows, K] in bf16, fp16 or fp32; w one matrix [N, K], or with `offsets` (int32 [G+1])
    G of them: rows offsets[g] .. offsets[g+1] of out belong to group g.  swiglu: w holds 2N
    rows, gate then up, and out = silu(gate) * up.  `index` (int32 [M]) with index_div names
    the rows of a: r = index[p] // index_div; without it r = p.  Rows of `out` in no group,
    or whose index is negative, are left as they were (a new `out` starts undefined there);
    `out` must not overlap an input.  A new `out` is of out_dtype, a's type if None.  There
    is no gradient: an `a` or `out` that wants one, or carries a tangent, is refused."""
    if not isinstance(w, Int4Weight):
        raise ValueError("w must be an Int4Weight")
    dev = gpu_tensor(a, "a", w.codes.get_device()).get_device()
    adt = dtype_of(a, "a")
    G = 0 if offsets is None else offsets.numel() - 1
    if a.dim() != 2 or a.shape[1] != w.K or G != w.G:
        raise ValueError(f"a {list(a.shape)} and {G} groups do not fit {w.G} matrices of "
                         f"{w.N} x {w.K}")
    if swiglu and w.N % 2:
        raise ValueError("swiglu needs an even number of rows of weights")
    N = w.N // 2 if swiglu else w.N
    M = rows = a.shape[0]
    for t, what in ((offsets, "offsets"), (index, "index")):
        if t is not None and gpu_tensor(t, what, dev).dtype != torch.int32:
            raise ValueError(f"{what} must be int32")
    if index is not None:
        index, M = index.contiguous(), index.numel()
    if max(rows, M) > B.MOE_INT_MAX or not B.fits(index_div):
        raise B.MoeError(B.MOE_EUNSUPPORTED, "moe_int4_matmul")
    _no_gradient("matmul", a, *(() if out is None else [out]))
    a, stride = row_major(a)
    if offsets is not None:
        offsets = offsets.contiguous()
    given = out is not None
    if not given:
        out_dtype = out_dtype or a.dtype
        if out_dtype not in DTYPES:
            raise ValueError(f"out_dtype must be bfloat16, float16 or float32, not {out_dtype}")
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    elif gpu_tensor(out, "out", dev).shape != (M, N):
        raise ValueError(f"out must have shape [{M}, {N}]")
    od = dtype_of(out, "out")
    if (N > 1 and out.stride(1) != 1) or (M > 1 and out.stride(0) < N):
        raise ValueError("the rows of out must be contiguous and apart")
    _matmul(a, B.Int4MatmulArgs(
        M, N, w.K, G, 1 if swiglu else 0, rows, a.data_ptr(), stride, adt,
        None if index is None else index.data_ptr(), int(index_div),
        None if offsets is None else offsets.data_ptr(), *w._args(), out.data_ptr(),
        out.stride(0) if M > 1 else N, od))
    if given:
        _written(out)
    return out


@on_its_device
def _matmul(a, args):
    st = _lib.moe_int4_matmul(args, stream_of(a))
    if st != B.MOE_OK:
        raise B.MoeError(st, "moe_int4_matmul")


class Int4Experts:
    """SwiGLU experts of a layer in 4 bits, one group for each slot: gate_up an Int4Weight
    [S, 2I, H] (gate rows, then up rows) and down one [S, H, I].  from_weights quantises
    floating weights slot by slot."""

    def __init__(self, gate_up: Int4Weight, down: Int4Weight):
        S, two_i, H = gate_up.G, gate_up.N, gate_up.K
        if not S or two_i % 2 or (down.G, down.N, down.K) != (S, H, two_i // 2):
            raise ValueError(f"down {[down.G, down.N, down.K]} does not fit gate_up "
                             f"{[S, two_i, H]}")
        if gate_up.device != down.device:
            raise ValueError(f"gate_up is on {gate_up.device}, down on {down.device}")
        self.gate_up, self.down = gate_up, down
        self.S, self.I, self.H = S, two_i // 2, H

    @classmethod
    def empty(cls, S: int, H: int, I: int, device, *, group: int = 128, zeros: bool = False,
              scale_dtype: torch.dtype = torch.bfloat16) -> "Int4Experts":
        kw = dict(group=group, zeros=zeros, scale_dtype=scale_dtype, device=device)
        return cls(Int4Weight.empty(S, 2 * I, H, **kw), Int4Weight.empty(S, H, I, **kw))

    @classmethod
    def from_weights(cls, gate, up, down, *, group: int = 128, zeros: bool = False,
                     scale_dtype: torch.dtype = torch.bfloat16) -> "Int4Experts":
        """gate, up [S, I, H] and down [S, H, I] in bf16, fp16 or fp32."""
        S, I, H = gate.shape
        e = cls.empty(S, H, I, gate.device, group=group, zeros=zeros, scale_dtype=scale_dtype)
        for s in range(S):
            e.load(s, gate[s], up[s], down[s])
        return e

    def load(self, slot: int, gate, up, down) -> None:
        """Quantises one expert's floating weights into a slot."""
        gu = self.gate_up[slot]
        if self.I % 16:  # the up rows begin inside a tile
            gu.load(torch.cat([gate, up]))
        else:
            gu.load(gate)
            gu.load(up, self.I)
        self.down[slot].load(down)

    def check(self, x, T: int) -> None:
        """Refuses token rows that are not [T, H] of a type that matmul takes, on the
        experts' device, or that want a gradient."""
        gpu_tensor(x, "x", self.gate_up.codes.get_device())
        dtype_of(x, "x")
        if tuple(x.shape) != (T, self.H):
            raise ValueError(f"x must have shape [{T}, {self.H}], not {list(x.shape)}")
        _no_gradient("Int4Experts", x)

    def rows(self, x, slot_offsets, perm, k: int) -> torch.Tensor:
        """The experts on the rows of a bucketing: token rows x [T, H] -> [T*k, H], row p from
        token perm[p] // k; rows that are in no slot are undefined.  The rows between the
        products and the result are rounded to x's type, half the bytes of float32 and the
        cheaper operand (float32 ones take three products): off by at most half a step each,
        2^-8 of a value in bf16."""
        self.check(x, x.shape[0])
        if perm.numel() > x.shape[0] * k:
            raise ValueError(f"perm holds {perm.numel()} values, more than the T*k = "
                             f"{x.shape[0] * k} assignments of x")
        h = matmul(x, self.gate_up, offsets=slot_offsets, index=perm, index_div=k, swiglu=True)
        return matmul(h, self.down, offsets=slot_offsets)

    def forward(self, x, slot_offsets, perm, sel_weight, pos=None) -> torch.Tensor:
        """x [T, H] -> [T, H] in x's type: the layer's experts and their weighted sum, from
        what moe_route wrote for the batch."""
        T, k = sel_weight.shape
        self.check(x, T)
        order = RowOrder(perm, T, k, pos)
        return combine(self.rows(x, slot_offsets, perm, k), order, sel_weight)
