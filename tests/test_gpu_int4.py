"""Products with 4-bit weights against float64.

Tolerance of a value: within a group of weights the sums run over a * (16 + code), K
products in float32 with magnitudes up to 31 |a|, and the correction (16 + zero) * sum a
adds two more roundings; the groups are then added with their scales.  Together at most
(K + 16) * 2^-23 of sum_i scale * 31 * |a_i| twice over (the sum and its correction), and
half a step of the output type."""
import pytest
import torch

from grouped_oracle import STEP, bucketing, rounding, silu, worst

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def random_weight(lead, N, K, group, zeros, scale_dtype, gen):
    codes = torch.randint(0, 16, (*lead, N, K), dtype=torch.uint8, generator=gen)
    n = -(-K // group)
    scale = (torch.rand(*lead, N, n, generator=gen) * 0.2 * K ** -0.5 + 1e-3).to(scale_dtype)
    zero = torch.randint(0, 16, (*lead, N, n), dtype=torch.uint8, generator=gen) if zeros else None
    cuda = lambda t: None if t is None else t.cuda()
    return cuda(codes), cuda(scale), cuda(zero)


def values(codes, scale, zero, group):
    """(weights, scales) in float64, one for each weight."""
    K = codes.shape[-1]
    wide = lambda t: t.double().repeat_interleave(group, dim=-1)[..., :K]
    z = 8.0 if zero is None else wide(zero)
    return (codes.double() - z) * wide(scale), wide(scale)


def reference(a, w, scale, swiglu, dtype):
    """(out, its bound) of one group."""
    a, K = a.double(), a.shape[1]
    N = w.shape[0] // (2 if swiglu else 1)
    t = lambda v: v.t().contiguous()
    y = a @ t(w)
    e = 2 * (K + 16) * STEP * (a.abs() @ t(31 * scale.abs()))
    if swiglu:
        g, u, eg, eu = y[:, :N], y[:, N:], e[:, :N], e[:, N:]
        y = silu(g) * u
        e = 1.1 * eg * (u.abs() + eu) + silu(g).abs() * eu + \
            (1.25 * g.abs() + 12) * 2.0 ** -24 * y.abs()
    return y, e + rounding(y.abs() + e, dtype)


SHAPES = [  # rows of the groups (None: dense, this many rows), N, K
    (1, 1, 1), (1, 33, 31), (5, 64, 128), (16, 48, 256), (17, 130, 384), (70, 96, 1000),
    ([1], 16, 32), ([1, 0, 2], 31, 129), ([16, 17, 0, 33], 64, 512), ([64, 65, 3], 50, 260),
    ([0, 130, 1, 1, 0], 128, 2304), ([0, 0], 40, 40), ([1] * 40, 256, 640),
]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("group,zeros,scale_dtype,swiglu", [
    (128, False, BF16, False), (64, True, FP16, True), (32, True, BF16, False),
    (32, False, FP16, True), (128, True, BF16, True), (64, False, BF16, False)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_products(shape, group, zeros, scale_dtype, swiglu, dtype):
    from resident_expert_routing_amd import int4
    counts, N, K = SHAPES[shape]
    gen = torch.Generator().manual_seed(shape)
    dense = isinstance(counts, int)
    lead = () if dense else (len(counts),)
    wide = 2 * N if swiglu else N
    codes, scale, zero = random_weight(lead, wide, K, group, zeros, scale_dtype, gen)
    w = int4.pack(codes, scale, zero, group=group)
    exact, sc = values(codes, scale, zero, group)
    assert torch.equal(w.dequantize(torch.float32).double(), exact.float().double())
    if dense:
        M, perm, offsets, k = counts, None, None, 1
        spans = [(None, 0, M)]
    else:
        k = 2
        perm, offsets = bucketing(counts, gen, tail=4)
        if perm.numel() % 2:
            perm = torch.cat([perm, torch.full((1,), -1, dtype=torch.int32)])
        M = perm.numel()
        e = offsets.tolist()
        spans = [(g, lo, hi) for g, (lo, hi) in enumerate(zip(e, e[1:])) if hi > lo]
        perm, offsets = perm.cuda(), offsets.cuda()
    a = (torch.randn(M // k, K, generator=gen) * 0.8).to(dtype).cuda()
    out = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    y = int4.matmul(a, w, offsets=offsets, index=perm, index_div=k, swiglu=swiglu, out=out)
    assert y is out
    for g, lo, hi in spans:
        rows = a if perm is None else a[(perm[lo:hi] // k).long()]
        at = () if g is None else (g,)
        want, tol = reference(rows, exact[at], sc[at], swiglu, dtype)
        ratio = worst(y[lo:hi], want, tol)
        print(f"group {g} rows {lo}..{hi}: {ratio:.3f}", flush=True)
        assert ratio <= 1
    assert (y[spans[-1][2] if spans else 0:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N,K", [(1, 1), (16, 128), (37, 300), (50, 97)])
def test_quantize(N, K, zeros, group, dtype):
    from resident_expert_routing_amd import int4
    gen = torch.Generator().manual_seed(N)
    w = (torch.randn(N, K, generator=gen) * torch.exp(torch.randn(N, 1, generator=gen))).to(dtype)
    if N > 3:
        w[2] = 0
    w = w.cuda()
    q = int4.quantize(w, group, zeros=zeros, scale_dtype=FP16)
    n = -(-K // group)
    padded = torch.zeros(N, n * group, device="cuda")
    padded[:, :K] = w.float()
    v = padded.view(N, n, group)
    lo, hi = v.amin(2).clamp(max=0), v.amax(2).clamp(min=0)
    want = ((hi - lo) / 15 if zeros else torch.maximum(hi, -lo) / 7).half()
    scale = q.scale.transpose(1, 2).reshape(-1, q.scale.shape[1])[:N, :n]
    assert torch.equal(scale, want)
    s = scale.float().unsqueeze(2)
    z = torch.full_like(s, 8.0)
    if zeros:
        z = torch.where(s > 0, torch.round(-lo.unsqueeze(2) / s).clamp(0, 15), z)
        got = q.zero.transpose(1, 2).reshape(-1, q.zero.shape[1])[:N, :n]
        assert torch.equal(got.float(), z.squeeze(2))
    codes = (torch.round(torch.where(s > 0, v / s, torch.zeros_like(v))) + z).clamp(0, 15)
    exact = ((codes - z) * s).reshape(N, -1)[:, :K]
    assert torch.equal(q.dequantize(), exact)
