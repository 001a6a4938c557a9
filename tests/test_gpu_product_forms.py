"""Every form of the grouped and 4-bit products against float64, at sizes that take it: each
test asserts the form first (product_forms has the rules)."""
import pytest
import torch

from grouped_oracle import STEP, Reference, bucketing, rounding, within, worst
from product_forms import int4_form, outer_form, rows_form, tile_heights, whole
from test_gpu_int4 import random_weight, reference, values

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32

# rows of the groups, on both sides of every tile height, alone and as the rest of a longer
# group; and many small groups, so that tiles are enough for the large form
COUNTS = [1, 63, 64, 65, 0, 127, 128, 129, 191, 192, 193, 255, 256, 257, 319, 320, 321, 383, 385,
          449, 512, 575, 640, 700] + [3, 0, 17] * 40


@pytest.mark.parametrize("K", [328, 331])  # whole pieces, and not; six stages and more
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("swiglu,across,by_token", [
    (False, False, False), (True, False, True), (False, True, True), (True, True, False),
    (False, False, True), (True, True, True)])
def test_large_tiles(swiglu, across, by_token, dtype, K):
    from resident_expert_routing_amd import grouped, rows
    G, N = len(COUNTS), 264 if swiglu else 520
    if K % 8:
        N += 3
    wide, k = (2 * N if swiglu else N), 2
    gen = torch.Generator().manual_seed(K + swiglu)
    perm, offsets = bucketing(COUNTS, gen, tail=4 + sum(COUNTS) % 2)
    M = perm.numel()
    esize = dtype.itemsize
    dma = whole(esize, K, wide if across else K)
    assert dma == (K % 8 == 0)
    for n, glu, lies in ((N, swiglu, across), (K, False, not across)):   # forward, rows' gradient
        form, R, blocks = rows_form(M, n, G, glu, lies, esize, dma)
        assert (form, blocks) == ("tiles", False)
        heights = {2, 4} if esize == 4 else {2, 4, 6, 8, 10} if dma else {2, 4, 8}
        assert tile_heights(COUNTS, R, esize, dma) == heights
    assert outer_form(M, wide, K, G, esize) == ("tiles", False)

    a = torch.randn(M // k if by_token else M, K, generator=gen).to(dtype).cuda()
    b = torch.randn(G, wide, K, generator=gen).mul_(1.5 * K ** -0.5)
    store = (b.transpose(1, 2).contiguous() if across else b).to(dtype).cuda()
    d = torch.randn(M, N, generator=gen).to(dtype).cuda()
    perm, offsets = perm.cuda(), offsets.cuda()
    view = lambda t: t.transpose(1, 2) if across else t
    index = torch.where(perm < 0, perm, perm // k) if by_token else None
    ref = Reference(a, view(store), offsets, index, M, swiglu, dtype, d, token_sum=by_token)

    kw = dict(index=perm, index_div=k) if by_token else {}
    with torch.no_grad():
        y = grouped.matmul(a, view(store), offsets, swiglu=swiglu, **kw)
    assert within(y, ref.out, ref.out_tol)
    a.requires_grad_(), store.requires_grad_()
    order = rows.RowOrder(perm, M // k, k) if by_token else None
    y2 = grouped.matmul(a, view(store), offsets, order=order, swiglu=swiglu)
    assert torch.equal(y, y2)
    da, db = torch.autograd.grad(y2, [a, store], d)
    print(f"y {worst(y, ref.out, ref.out_tol):.3f} da {worst(da, ref.da, ref.da_tol):.3f} "
          f"db {worst(view(db), ref.db, ref.db_tol):.3f}", flush=True)
    assert within(da, ref.da, ref.da_tol)
    assert within(view(db), ref.db, ref.db_tol)


@pytest.mark.parametrize("dtype,K,swiglu,across", [(BF16, 136, True, False), (FP16, 136, False, True),
                                                   (BF16, 75, True, True), (FP32, 68, True, False)])
def test_rows_in_xcd_blocks(dtype, K, swiglu, across):
    """Long groups over many columns, whose tiles are dealt to the XCDs in blocks."""
    from resident_expert_routing_amd import grouped
    counts = [30001, 0, 20479, 14000, 1]
    N = 1301 if swiglu else 2584
    if dtype == FP32:
        counts, N = [9001, 0, 5000, 12000], 1301
    gen = torch.Generator().manual_seed(K)
    perm, offsets = bucketing(counts, gen, tail=700)
    M, G, wide = perm.numel(), len(counts), 2 * N if swiglu else N
    if K % 8 == 0:
        wide = wide // 16 * 16
        N = wide // 2 if swiglu else wide
    dma = whole(dtype.itemsize, K, wide if across else K)
    assert rows_form(M, N, G, swiglu, across, dtype.itemsize, dma)[::2] == ("tiles", True)
    a = torch.randn(M, K, generator=gen).to(dtype).cuda()
    b = (torch.randn(G, wide, K, generator=gen) * K ** -0.5).to(dtype).cuda()
    if across:
        b = b.transpose(1, 2).contiguous().transpose(1, 2)
    perm, offsets = perm.cuda(), offsets.cuda()
    y = grouped.matmul(a, b, offsets, index=perm, swiglu=swiglu)
    ref = Reference(a, b, offsets, perm, M, swiglu, dtype)
    assert within(y, ref.out, ref.out_tol)
    assert not y[int(offsets[-1]):].any()


@pytest.mark.parametrize("dtype,L,R,side", [(BF16, 4096, 3968, None), (FP16, 4088, 3976, "right"),
                                            (BF16, 3999, 4001, "left"), (FP32, 2044, 1956, "right")])
def test_outer_tiles_in_xcd_blocks(dtype, L, R, side):
    from resident_expert_routing_amd import grouped
    G, k = 32, 2
    counts = [256 + (37 * g) % 81 for g in range(G - 2)] + [0, 700]
    gen = torch.Generator().manual_seed(L)
    perm, offsets = bucketing(counts, gen, tail=sum(counts) % 2)
    M = perm.numel()
    assert outer_form(M, L, R, G, dtype.itemsize) == ("tiles", True)
    dev = lambda t: t.to(dtype).cuda()
    left = dev(torch.randn(M // k if side == "left" else M, L, generator=gen))
    right = dev(torch.randn(M // k if side == "right" else M, R, generator=gen))
    perm, offsets = perm.cuda(), offsets.cuda()
    of = lambda s: (perm, k) if side == s else (None, 1)
    got = grouped._outer(left, *of("left"), right, *of("right"), offsets, M)
    edges = offsets.tolist()
    for g in range(G):
        p = torch.arange(edges[g], edges[g + 1], device="cuda")
        named = perm[p].long() // k
        x = left[named if side == "left" else p].double().t().contiguous()
        y = right[named if side == "right" else p].double()
        want = x @ y
        tol = p.numel() * STEP * (x.abs() @ y.abs())
        assert within(got[g], want, tol + rounding(want.abs() + tol, dtype))


# rows of the groups (one number: dense), columns, the form
INT4 = [(1, 64, "few"), (40, 128, "few"), ([1, 0, 3], 64, "few"),
        (130, 1024, "mid"), ([2] * 9, 1024, "mid"),
        (700, 2100, "thin"), ([1, 0, 2] * 120, 300, "thin"), ([9, 40, 3, 0] * 16, 1030, "thin"),
        (90, 32768, "wide"), ([70, 31, 0, 65, 1] * 65, 257, "wide")]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("group,zeros,swiglu,K", [(128, False, True, 300), (64, True, True, 256),
                                                  (32, True, False, 170), (128, True, False, 384)])
@pytest.mark.parametrize("at", range(len(INT4)))
def test_int4_forms(at, group, zeros, swiglu, K, dtype):
    from resident_expert_routing_amd import int4
    counts, N, want = INT4[at]
    if want == "wide" and isinstance(counts, int) and not swiglu:
        N *= 2
    dense = isinstance(counts, int)
    G = 0 if dense else len(counts)
    gen = torch.Generator().manual_seed(at)
    codes, scale, zero = random_weight((G,) if G else (), 2 * N if swiglu else N, K, group, zeros,
                                       BF16, gen)
    w = int4.pack(codes, scale, zero, group=group)
    exact, sc = values(codes, scale, zero, group)
    del codes
    perm, offsets = (None, None) if dense else bucketing(counts, gen, tail=3)
    M = counts if dense else perm.numel()
    assert int4_form(M, N, G, swiglu) == want
    a = torch.randn(M, K, generator=gen).to(dtype).cuda()
    if dense:
        spans = [((), 0, M)]
    else:
        perm, offsets = perm.cuda(), offsets.cuda()
        e = offsets.tolist()
        spans = [((g,), lo, hi) for g, (lo, hi) in enumerate(zip(e, e[1:])) if hi > lo]
    out = torch.full((M, N), 5.0, dtype=dtype, device="cuda")
    int4.matmul(a, w, offsets=offsets, index=perm, swiglu=swiglu, out=out)
    for g, lo, hi in spans:
        x = a if dense else a[perm[lo:hi].long()]
        y, tol = reference(x, exact[g], sc[g], swiglu, dtype)
        assert within(out[lo:hi], y, tol)
    assert (out[spans[-1][2]:] == 5).all()


@pytest.mark.parametrize("group", [32, 64, 128])
def test_experts_keep_their_weights_to_a_step(group):
    """What Int4Experts stores, with zero points and without: off by at most half a step of the
    group's scale, and where the last code cuts, by what bf16 rounded the scale down, 2^-8 of
    15 steps, more.  Without zero points 7 (1 + 2^-8) steps still round to 7."""
    from resident_expert_routing_amd import int4
    gen = torch.Generator().manual_seed(group)
    S, H, I = 3, 320, 40
    gate, up = (torch.randn(S, I, H, generator=gen).cuda() for _ in range(2))
    down = torch.randn(S, H, I, generator=gen).cuda()
    for zeros in (False, True):
        ex = int4.Int4Experts.from_weights(gate, up, down, group=group, zeros=zeros)
        for q, w in ((ex.gate_up, torch.cat([gate, up], 1)), (ex.down, down)):
            scale = q.scale.double().transpose(-1, -2).reshape(S, -1, q.scale.shape[-2])
            step = scale.repeat_interleave(group, -1)[:, :w.shape[1], :w.shape[2]]
            most = 0.5 + 15 * 2.0 ** -8 if zeros else 0.5
            off = (q.dequantize().double() - w.double()).abs() / step
            print(f"group {group} zeros {zeros}: {float(off.max()):.4f} of a step", flush=True)
            assert float(off.max()) <= most + 1e-5
