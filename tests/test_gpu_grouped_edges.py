"""Grouped products at the edges: what no row may touch, layouts, many groups, long groups,
sizes past 32 bits, other streams and graphs, refusals, and the layer that uses them."""
import pytest
import torch
from torch.autograd import forward_ad

from grouped_oracle import Reference, bucketing, silu, within

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def case(counts, N, K, dtype, seed=0, swiglu=False, tail=5):
    gen = torch.Generator().manual_seed(seed)
    _, offsets = bucketing(counts, gen)
    M, wide = sum(counts) + tail, 2 * N if swiglu else N
    a = torch.randn(M, K, generator=gen).to(dtype).cuda()
    b = (torch.randn(len(counts), wide, K, generator=gen) * K ** -0.5).to(dtype).cuda()
    d = torch.randn(M, N, generator=gen).to(dtype).cuda()
    return a, b, offsets.cuda(), d


def check(a, b, offsets, d, swiglu=False, index=None, M=None, **kw):
    """Forward and both gradients against float64."""
    from resident_expert_routing_amd import grouped
    ref = Reference(a.detach(), b.detach(), offsets, index, a.shape[0] if M is None else M, swiglu,
                    a.dtype, d, token_sum=index is not None)
    y = grouped.matmul(a, b, offsets, swiglu=swiglu, **kw)
    assert within(y.detach(), ref.out, ref.out_tol)
    da, db = torch.autograd.grad(y, [a, b], d)
    assert within(da, ref.da, ref.da_tol)
    assert within(db, ref.db, ref.db_tol)


@pytest.mark.parametrize("dtype,K,N", [(BF16, 72, 136), (FP16, 67, 131), (FP32, 40, 33)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_other_rows_do_not_matter(dtype, K, N, swiglu):
    """Infinities and NaN in rows of other groups, or of none, and in their gradients."""
    from resident_expert_routing_amd import grouped
    counts = [5, 70, 0, 3, 66]
    a, b, offsets, d = case(counts, N, K, dtype, swiglu=swiglu)
    edges = offsets.tolist()
    clean = slice(edges[1], edges[2])
    bad = torch.ones(a.shape[0], dtype=torch.bool, device="cuda")
    bad[clean] = False
    a2, d2, b2 = a.clone(), d.clone(), b.clone()
    a2[bad], d2[bad] = float("nan"), float("inf")
    b2[[0, 2, 3, 4]] = float("inf")
    outs = []
    for x, w, g in ((a, b, d), (a2, b2, d2)):
        x, w = x.requires_grad_(), w.requires_grad_()
        y = grouped.matmul(x, w, offsets, swiglu=swiglu)
        da, db = torch.autograd.grad(y, [x, w], g)
        outs.append((y.detach(), da, db))
    (y, da, db), (y2, da2, db2) = outs
    assert torch.equal(y[clean], y2[clean]) and torch.equal(da[clean], da2[clean])
    assert torch.equal(db[1], db2[1])
    assert not db2[2].any()                                        # the group without rows
    rest = slice(edges[-1], None)
    assert not y2[rest].any() and not da2[rest].any()              # rows of no group: zero


@pytest.mark.parametrize("K,N,dtype", [(64, 128, BF16), (65, 50, FP16), (24, 20, FP32)])
def test_rows_of_no_group(K, N, dtype):
    """Before the first group and behind the last: zero in a new out, left in the caller's;
    nothing beside the rows of a strided out is written."""
    from resident_expert_routing_amd import grouped
    a, b, offsets, _ = case([40, 0, 80], N, K, dtype, tail=300)
    offsets = offsets + 200
    M = a.shape[0]
    y = grouped.matmul(a, b, offsets)
    out = torch.full((M + 2, N + 6), 3.0, dtype=dtype, device="cuda")
    view = out[1:-1, 3:3 + N]
    assert grouped.matmul(a, b, offsets, out=view) is view
    live = torch.zeros(M, dtype=torch.bool, device="cuda")
    live[200:320] = True
    assert torch.equal(view[live], y[live]) and y[live].any()
    assert not y[~live].any() and (view[~live] == 3).all()
    view[live] = 3
    assert (out == 3).all()
    # offsets past the rows are cut
    cut = grouped.matmul(a[:250], b, offsets)
    assert torch.equal(cut[:240], y[:240]) and cut.shape[0] == 250


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_layouts(dtype):
    """Rows at odd addresses and distances, matrices as slices, transposed or shared, and a
    gradient that is broadcast."""
    a, b, offsets, d = case([33, 7, 129], 72, 96, dtype, seed=1)
    wide = torch.zeros(a.shape[0], 140, dtype=dtype, device="cuda")
    odd = wide[:, 21:117].copy_(a).requires_grad_()
    check(odd, b.requires_grad_(), offsets, d)
    big = torch.zeros(3, 80, 101, dtype=dtype, device="cuda")
    for view in (big[:, 3:75, 5:101], big[:, 3:75, 4:100]):
        check(a.requires_grad_(), view.copy_(b.detach()).detach().requires_grad_(), offsets, d)
    shared = b.detach()[:1].clone().requires_grad_()
    one = b.detach()[:1].expand(3, -1, -1).requires_grad_()
    check(a, one, offsets, d)
    from resident_expert_routing_amd import grouped
    y = grouped.matmul(a, shared.expand(3, -1, -1), offsets)
    ref = Reference(a.detach(), shared.detach().expand(3, -1, -1), offsets, None, a.shape[0], False,
                    dtype, d)
    g, = torch.autograd.grad(y, shared, d)
    # autograd adds the three groups' gradients in the element type: two roundings more
    total, tol = ref.db.sum(0), ref.db_tol.sum(0)
    tol = tol + 2 * torch.finfo(dtype).eps * (ref.db.abs().sum(0) + tol)
    assert within(g[0], total, tol)
    x = a.detach().requires_grad_()
    grouped.matmul(x, b.detach(), offsets).sum().backward()
    ones = torch.ones_like(d)
    ref = Reference(x.detach(), b.detach(), offsets, None, x.shape[0], False, dtype, ones)
    assert within(x.grad, ref.da, ref.da_tol)


@pytest.mark.parametrize("G", [257, 1000, 4097])
def test_many_groups(G):
    from resident_expert_routing_amd import grouped
    gen = torch.Generator().manual_seed(G)
    counts = (torch.rand(G, generator=gen) < 0.1).int() * torch.randint(1, 9, (G,), generator=gen)
    counts[-1] = 3
    a, b, offsets, d = case(counts.tolist(), 40, 48, BF16, tail=70)
    check(a.requires_grad_(), b.requires_grad_(), offsets, d)
    y = grouped.matmul(a.detach(), b.detach(), offsets)
    assert not y[int(offsets[-1]):].any()


@pytest.mark.parametrize("dtype,N,K", [(BF16, 64, 72), (FP16, 35, 41)])
def test_a_long_group_named_by_token(dtype, N, K):
    """More rows than the outer product's table holds, several times over, some of which
    name no token."""
    from resident_expert_routing_amd import grouped, rows
    T, k = 3001, 2
    gen = torch.Generator().manual_seed(3)
    perm = torch.randperm(T * k, generator=gen).int()
    perm[-100:] = -1
    offsets = torch.tensor([0, 1, 5400, T * k - 100], dtype=torch.int32)
    a = torch.randn(T, K, generator=gen).to(dtype).cuda().requires_grad_()
    b = (torch.randn(3, N, K, generator=gen) * K ** -0.5).to(dtype).cuda().requires_grad_()
    d = torch.randn(T * k, N, generator=gen).to(dtype).cuda()
    perm, offsets = perm.cuda(), offsets.cuda()
    order = rows.RowOrder(perm, T, k)
    index = torch.where(perm < 0, perm, perm // k)
    check(a, b, offsets, d, index=index, M=T * k, order=order)
    # rows inside a group whose index names nothing
    holes = index.clone()
    holes[2:5000:7] = -1
    holes[3:5000:11] = T
    ref = Reference(a.detach(), b.detach(), offsets, holes, T * k, False, dtype, d)
    d2 = d.clone()
    d2[(holes < 0) | (holes >= T)] = float("nan")
    y = grouped.matmul(a.detach(), b, offsets, index=holes)
    assert within(y.detach(), ref.out, ref.out_tol)
    db, = torch.autograd.grad(y, b, d2)
    assert within(db, ref.db, ref.db_tol)


def test_sizes_past_32_bits():
    """Matrices, and an out, of more than 2^31 elements."""
    from resident_expert_routing_amd import grouped
    G, N, K = 130, 4352, 4096
    b = torch.empty(G, N, K, dtype=BF16, device="cuda")
    b[-1].normal_(std=0.02)
    a = torch.randn(70, K, device="cuda").to(BF16)
    offsets = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = 70
    assert b.numel() > 2 ** 31
    ref = Reference(a, b[-1:], torch.tensor([0, 70]), None, 70, False, BF16)
    assert within(grouped.matmul(a, b, offsets), ref.out, ref.out_tol)
    b2 = b.transpose(1, 2).contiguous().transpose(1, 2)
    del b
    assert within(grouped.matmul(a, b2, offsets), ref.out, ref.out_tol)
    db = grouped._outer(a, None, 1, a, None, 1, offsets, 70)  # [130, 4096, 4096]
    assert db.numel() > 2 ** 31 and not db[:-1].any()
    want = a.double().t().contiguous() @ a.double()
    tol = 70 * 2.0 ** -23 * (a.double().abs().t().contiguous() @ a.double().abs()) + \
        want.abs() * 2.0 ** -8
    assert within(db[-1], want, tol + 1e-30)
    del b2, db
    M, N, K = 70000, 32768, 64
    a, b = torch.randn(M, K, device="cuda").to(BF16), torch.randn(1, N, K, device="cuda").to(BF16)
    y = grouped.matmul(a, b, torch.tensor([0, M], dtype=torch.int32, device="cuda"))
    some = torch.tensor([0, 65535, 65536, M - 1], device="cuda")
    ref = Reference(a[some], b, torch.tensor([0, 4]), None, 4, False, BF16)
    assert within(y[some], ref.out, ref.out_tol)


def test_no_rows():
    from resident_expert_routing_amd import grouped, rows
    b = torch.randn(3, 16, 24, device="cuda", requires_grad=True)
    offsets = torch.zeros(4, dtype=torch.int32, device="cuda")
    a = torch.empty(0, 24, device="cuda", requires_grad=True)
    for kw in ({}, dict(swiglu=True),
               dict(order=rows.RowOrder(torch.empty(0, dtype=torch.int32, device="cuda"), 0, 4))):
        y = grouped.matmul(a, b, offsets, **kw)
        da, db = torch.autograd.grad(y, [a, b], torch.zeros_like(y))
        assert y.shape == (0, 8 if kw.get("swiglu") else 16) and da.shape == a.shape
        assert db.shape == b.shape and not db.any()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_saturating_gates_backward(dtype):
    """Gates from -90 to 90: the gradient is that of the formula, and finite."""
    from resident_expert_routing_amd import grouped
    n = 181
    g = torch.arange(n, device="cuda").float() - 90
    pre = torch.cat([g, torch.linspace(-3, 3, n, device="cuda")])[None]
    d = torch.linspace(0.5, 2, n, device="cuda")[None].to(dtype)
    got = grouped._swiglu_backward(d, pre).double()
    gd, u, dd = pre[:, :n].double(), pre[:, n:].double(), d.double()
    s = torch.sigmoid(gd)
    want = torch.cat([dd * u * (s + gd * s * (1 - s)), dd * silu(gd)], 1)
    # exp's argument 1.25 |g| units of 2^-24, the exponential and reciprocal 2 each, eight
    # products and sums; s + v (1 - s) cancels, so its bound is that of its terms
    big = torch.cat([(dd * u).abs() * (s + (gd * s * (1 - s)).abs()), (dd * silu(gd)).abs()], 1)
    tol = big * (1.25 * gd.abs().repeat(1, 2) + 12) * 2.0 ** -24
    eps = torch.finfo(dtype)
    tol = tol + (want.abs() + tol) * eps.eps / 2 + max(eps.smallest_normal * eps.eps, 2.0 ** -122)
    assert within(got, want, tol)


def test_gradient_against_differences():
    from resident_expert_routing_amd import grouped
    a, b, offsets, d = case([9, 0, 21], 12, 10, FP32, swiglu=True, tail=2)
    a, b = (a * 0.5).requires_grad_(), b.requires_grad_()
    f = lambda x, w: (grouped.matmul(x, w, offsets, swiglu=True).double() * d.double()).sum()
    ga, gb = torch.autograd.grad(f(a, b), [a, b])
    gen = torch.Generator(device="cuda").manual_seed(5)
    for t, g, at in ((a, ga, 0), (b, gb, 1)):
        for _ in range(4):
            v = torch.randn(t.shape, generator=gen, device="cuda")
            h = 2.0 ** -7
            with torch.no_grad():
                lo, hi = [a, b], [a, b]
                lo[at], hi[at] = t - h * v, t + h * v
                slope = float(f(*hi) - f(*lo)) / (2 * h)
            # the difference is off by h^2 / 6 of the third derivative, some tens of |v|^3 here,
            # and by float32 rounding of 360 values over 2 h
            assert abs(slope - float((g.double() * v).sum())) <= 0.02 * float(g.norm() * v.norm())


def test_kept_order_and_offsets():
    """The next routing may write over offsets and perm before the backward pass; rows and
    matrices that are written over are refused."""
    from resident_expert_routing_amd import grouped, rows
    gen = torch.Generator().manual_seed(8)
    T, k = 50, 2
    perm, offsets = bucketing([30, 50, 20], gen)
    perm, offsets = perm.cuda(), offsets.cuda()
    a = torch.randn(T, 32, generator=gen).to(BF16).cuda().requires_grad_()
    b = torch.randn(3, 16, 32, generator=gen).to(BF16).cuda().requires_grad_()
    d = torch.randn(T * k, 16, generator=gen).to(BF16).cuda()
    def run(spoil, pos=None):
        y = grouped.matmul(a, b, offsets, order=rows.RowOrder(perm, T, k, pos))
        if spoil:
            perm.copy_(perm.flip(0)), offsets.fill_(7)
            if pos is not None:
                pos.zero_()
        return torch.autograd.grad(y, [a, b], d)
    keep = perm.clone(), offsets.clone()
    want = run(False)
    for pos in (None, rows.RowOrder(perm, T, k).pos.clone()):
        got = run(True, pos)
        perm.copy_(keep[0]), offsets.copy_(keep[1])
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    x = a.detach() * 1
    y = grouped.matmul(x, b, offsets, order=rows.RowOrder(perm, T, k))
    x.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.backward(d)


def test_refusals():
    from resident_expert_routing_amd import grouped, rows
    a, b, offsets, d = case([10, 20], 16, 24, BF16)
    bad = [
        dict(a=a.float()), dict(a=a.int()), dict(b=b[0]), dict(b=b[:1]), dict(b=b[:, :, :20]),
        dict(offsets=offsets.long()), dict(offsets=offsets[:1]), dict(offsets=offsets.cpu()),
        dict(b=b.cpu()), dict(a=a[0]), dict(b=b[:, :15], swiglu=True),
        dict(index=offsets, order=rows.RowOrder(offsets, 3, 1)), dict(index=offsets.long()),
        dict(order=rows.RowOrder(torch.arange(6, dtype=torch.int32, device="cuda"), 3, 2)),
        dict(out=torch.empty(35, 15, dtype=BF16, device="cuda")),
        dict(out=torch.empty(35, 16, dtype=FP16, device="cuda")),
        dict(out=torch.empty(16, 35, dtype=BF16, device="cuda").t()),
        dict(out=torch.empty(35, 16, dtype=BF16, device="cuda").requires_grad_()),
    ]
    for kw in bad:
        with pytest.raises(ValueError):
            grouped.matmul(**(dict(a=a, b=b, offsets=offsets) | kw))
    with pytest.raises(RuntimeError, match="moe_grouped_matmul"):
        grouped.matmul(a, b, offsets, index=torch.zeros(4, dtype=torch.int32, device="cuda"),
                       index_div=0)
    leaf = a.clone().requires_grad_()
    with pytest.raises(ValueError, match="order"):
        grouped.matmul(leaf, b, offsets, index=torch.arange(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="out"):
        grouped.matmul(leaf, b, offsets, out=torch.empty(35, 16, dtype=BF16, device="cuda"))
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(a, torch.ones_like(a))
        with pytest.raises(ValueError, match="tangent"):
            grouped.matmul(dual, b, offsets)
    y = grouped.matmul(leaf, b, offsets)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(y.sum(), leaf, create_graph=True)
    with pytest.raises(ValueError):
        grouped.GroupedExperts(b, b)


def test_a_given_out_counts_as_changed():
    from resident_expert_routing_amd import grouped
    a, b, offsets, d = case([10, 20], 16, 24, FP32)
    w = torch.randn(16, 4, device="cuda", requires_grad=True)
    buf = torch.zeros(35, 16, device="cuda")
    y = buf @ w
    grouped.matmul(a, b, offsets, out=buf)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.sum().backward()


@pytest.mark.parametrize("swiglu", [False, True])
def test_captured_and_replayed(swiglu):
    """Forward and backward in a graph: each replay against eager calls on what its inputs
    hold by then, with work of the program's own between them."""
    from resident_expert_routing_amd import grouped, rows
    T, k, K, N = 96, 2, 64, 48
    gen = torch.Generator().manual_seed(4)
    a = torch.randn(T, K, generator=gen).to(BF16).cuda()
    b = torch.randn(4, 2 * N if swiglu else N, K, generator=gen).to(BF16).cuda()
    d = torch.randn(T * k, N, generator=gen).to(BF16).cuda()
    orders = [[t.cuda() for t in bucketing(c, gen)] for c in ([10, 100, 0, 82], [0, 1, 190, 1],
                                                              [48] * 4)]
    perm, offsets = orders[0][0].clone(), orders[0][1].clone()

    def step(a, b):
        a, b = a.detach().requires_grad_(), b.detach().requires_grad_()
        y = grouped.matmul(a, b, offsets, order=rows.RowOrder(perm, T, k), swiglu=swiglu)
        return (y.detach(), *torch.autograd.grad(y, [a, b], d))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a, b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step(a, b)
    for i, (p, o) in enumerate(orders):
        perm.copy_(p), offsets.copy_(o)
        a.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in kept]
        want = step(a, b)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w), i


def test_two_streams():
    from resident_expert_routing_amd import grouped
    sets = [case([60, 0, 90, 200], 136, 128, BF16, seed=s, swiglu=True) for s in range(2)]
    def step(a, b, offsets, d):
        a, b = a.detach().requires_grad_(), b.detach().requires_grad_()
        y = grouped.matmul(a, b, offsets, swiglu=True)
        return (y.detach(), *torch.autograd.grad(y, [a, b], d))
    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for i, (s, stream) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(stream):
                got[i].append(step(*s))
    torch.cuda.synchronize()
    for i, runs in enumerate(got):
        for r in runs:
            assert all(torch.equal(x, y) for x, y in zip(r, want[i]))


@pytest.mark.parametrize("T,H,E,k,I,S,resident", [(8, 256, 16, 4, 128, 10, 10), (1, 64, 8, 2, 32, 6, 3),
                                                  (200, 256, 16, 4, 96, 9, 9)])
def test_layer(T, H, E, k, I, S, resident):
    """Routing, the experts and combine, with gradients to all that learns, against the same
    chain in float64 from the routing's own picks and weights."""
    from test_gpu_int8 import routed
    from resident_expert_routing_amd import grouped
    from resident_expert_routing_amd import runtime as R
    buf, x, (wg, wu, wd), args = routed(T, H, E, k, I, S, resident, T)
    gu = torch.cat([wg, wu], 1).to(BF16).requires_grad_()
    dn = wd.to(BF16).requires_grad_()
    x = x.requires_grad_()
    ex = grouped.GroupedExperts(gu, dn)
    sel = buf.sel_weight.clone().requires_grad_()
    out = ex.forward(x, buf.slot_offsets, buf.perm, sel)
    d = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    grads = torch.autograd.grad(out, [x, gu, dn, sel], d)

    off, perm = buf.slot_offsets.tolist(), buf.perm.long()
    leaves = [t.detach().double().requires_grad_() for t in (x, gu, dn, sel)]
    xd, gud, dnd, wd64 = leaves
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for s in range(S):
        p = perm[off[s]:off[s + 1]]
        if p.numel():
            z = xd[p // k] @ gud[s].t()
            h = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
            want = want.index_add(0, p // k, (h @ dnd[s].t()) * wd64.view(-1)[p, None])
    ref = torch.autograd.grad(want, leaves, d.double()) if want.requires_grad else \
        [torch.zeros_like(t) for t in leaves]
    # relative L2: each stage rounds to bf16, at most 2^-9 of a value (its rms 2^-9 / sqrt 3):
    # out h, y and itself; the gradients d, dy, dh, z and dz beside
    for name, g, w, n in (("out", out, want, 3), ("x", grads[0], ref[0], 8),
                          ("gate_up", grads[1], ref[1], 8), ("down", grads[2], ref[2], 6),
                          ("weight", grads[3], ref[3], 6)):
        g, w = g.detach().double(), w.detach()
        if not w.any():
            assert not g.any()
            continue
        rel = float((g - w).norm() / w.norm())
        print(f"{name}: {rel:.2e}", flush=True)
        assert rel <= n * 2.0 ** -9, name
    hist = torch.zeros(E, dtype=torch.float64, device="cuda")
    step = R.layer_step_grouped(buf, x.detach(), args[0], None, args[1], hist, ex)
    assert torch.equal(step, out) and float(hist.sum()) > 0
    for wrong in (x.detach()[:, :-1], x.detach().float(), torch.cat([x.detach()] * 2)):
        before = hist.clone()
        with pytest.raises(ValueError):
            R.layer_step_grouped(buf, wrong, args[0], None, args[1], hist, ex)
        assert torch.equal(hist, before)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("counts,N,K", [([1, 0, 2], 40, 96), ([70, 20], 33, 65), ([300, 4, 90] * 20, 520, 64),
                                        ([300, 4, 90] * 20, 517, 67)])
def test_rows_left_in_float32(counts, N, K, dtype):
    """An out of float32 holds what the rounded one is rounded from, in every form."""
    from resident_expert_routing_amd import grouped
    for across in (False, True):
        a, b, offsets, _ = case(counts, N, K, dtype, swiglu=False)
        if across:
            b = b.transpose(1, 2).contiguous().transpose(1, 2)
        M = a.shape[0]
        wide = torch.full((M, N), 9.0, device="cuda")
        grouped._products(a, grouped._matrices(b), offsets, None, 1, M, N, False, wide, True, False)
        assert torch.equal(wide.to(dtype), grouped.matmul(a, b, offsets))
        ref = Reference(a, b, offsets, None, M, False, FP32)
        assert within(wide, ref.out, ref.out_tol)


@pytest.mark.parametrize("dtype,N,K", [(BF16, 128, 192), (FP16, 70, 130), (FP32, 100, 64), (FP32, 33, 70)])
@pytest.mark.parametrize("across", [False, True])
def test_long_groups_of_small_matrices(dtype, N, K, across):
    """The rows of a group are summed in parts, through a workspace."""
    from resident_expert_routing_amd import binding as B
    from resident_expert_routing_amd import grouped
    counts = [5000, 0, 9001, 3]
    a, b, offsets, d = case(counts, N, K, dtype, seed=2)
    M = a.shape[0]
    assert B.moe_grouped_outer_ws_bytes(M, N, K, 4, grouped.dtype_of(a, "a")) > 0
    if across:
        b = b.transpose(1, 2).contiguous().transpose(1, 2)
    d[14004:] = float("nan")                              # rows of no group
    a, b = a.requires_grad_(), b.detach().requires_grad_()
    ref = Reference(a.detach(), b.detach(), offsets, None, M, False, dtype, d)
    db, = torch.autograd.grad(grouped.matmul(a, b, offsets), b, d)
    assert within(db, ref.db, ref.db_tol)
    again, = torch.autograd.grad(grouped.matmul(a, b, offsets), b, d)
    assert torch.equal(db, again)


def test_experts_that_do_not_fit():
    """Matrices of two types or places, or with a tangent, and buffers elsewhere are refused
    before the demand is counted, also where they came to differ after they were given."""
    from test_gpu_int8 import routed
    from resident_expert_routing_amd import grouped
    from resident_expert_routing_amd import runtime as R
    buf, x, (wg, wu, wd), args = routed(8, 64, 8, 2, 32, 6, 6, 0)
    gu, dn = torch.cat([wg, wu], 1).to(BF16), wd.to(BF16)
    for bad in ((gu, dn.float()), (gu.float(), dn), (gu, dn.to(FP16)), (gu, dn.cpu()), (gu.cpu(), dn),
                (gu.int(), dn.int()), (gu[0], dn), (gu, dn[0]),
                (gu, dn.transpose(1, 2))):
        with pytest.raises(ValueError):
            grouped.GroupedExperts(*bad)
    hist = torch.zeros(8, dtype=torch.float64, device="cuda")
    step = lambda ex, buf=buf: R.layer_step_grouped(buf, x, args[0], None, args[1], hist, ex)
    for which in range(2):
        pair = [torch.nn.Parameter(t.clone()) for t in (gu, dn)]
        ex = grouped.GroupedExperts(*pair)
        for new in (lambda t: t.float(), lambda t: t.cpu()):
            keep = pair[which].data
            pair[which].data = new(keep)
            with pytest.raises(ValueError):
                step(ex)
            pair[which].data = keep
        with forward_ad.dual_level():
            pair[which] = forward_ad.make_dual(pair[which].detach(), torch.ones_like(pair[which]))
            with pytest.raises(ValueError, match="tangent"):
                step(grouped.GroupedExperts(*pair))
    with pytest.raises(ValueError, match="GPU"):
        step(grouped.GroupedExperts(gu.cpu(), dn.cpu()))
    ex = grouped.GroupedExperts(gu, dn)
    with pytest.raises(ValueError):
        step(ex, R.LayerBuffers(8, 64, 8, 2, 32, 6, torch.device("cpu")))
    assert not hist.any()
    want = step(ex)
    assert want.shape == x.shape and hist.any()
    # a model may be made on the host and moved as a whole
    pair = [torch.nn.Parameter(t.cpu()) for t in (gu, dn)]
    ex = grouped.GroupedExperts(*pair)
    for t in pair:
        t.data = t.data.cuda()
    assert torch.equal(step(ex), want)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_low_gates(dtype):
    """Gates from -64 to -173, in a product and in its gradient, with ups and gradients so large
    that the value is a normal number: it keeps it."""
    from resident_expert_routing_amd import grouped
    f = torch.finfo(dtype)
    g = -torch.arange(64, 174, device="cuda").float()
    n = g.numel()
    # exp's argument 1.25 |g| units of 2^-24; the exponentials, reciprocal and products 12
    f32 = (1.25 * g.double().abs() + 12) * 2.0 ** -24
    small = f.smallest_normal * 1.01
    checked = 0
    for u, d in ((1e38, 1.0), (3e38, 0.5), (1e19, 1e19), (0.25, 3e38), (1e-2, 1e38), (-1e38, 1e-2)):
        us, ds = torch.full((n,), u, device="cuda"), torch.full((1, n), d, device="cuda").to(dtype)
        gd, ud, dd = g.double(), us.double(), ds.double()
        e = torch.exp(gd)
        s = e / (1 + e)
        want = torch.cat([dd * ud * (s + gd * s / (1 + e)), dd * gd * s], 1)
        got = grouped._swiglu_backward(ds, torch.cat([g, us])[None]).double()
        tol = want.abs() * (f32.repeat(2) + f.eps / 2 * 1.0001)
        normal = (want.abs() >= small) & (want.abs() <= f.max / 1.01)
        print(f"u {u} d {d}: {int(normal[:, :n].sum())} and {int(normal[:, n:].sum())} normal values, "
              f"worst {float(((got - want).abs() / tol)[normal].nan_to_num(9).max()):.3f}", flush=True)
        assert ((got - want).abs() <= tol)[normal].all()
        checked += int(normal.sum())
    assert checked > 3 * n
    # the product itself: gates and ups that are one number each
    up = 2.0 ** 127 * 1.5
    a = torch.stack([g, torch.ones_like(g)], 1).to(dtype)
    b = torch.tensor([[[1.0, 0.0], [0.0, up]]], device="cuda").to(dtype)
    y = grouped.matmul(a, b, torch.tensor([0, n], dtype=torch.int32, device="cuda"), swiglu=True)
    ad = a.double()
    e = torch.exp(ad[:, 0])
    want = ad[:, 0] * e / (1 + e) * float(b[0, 1, 1])
    ok = (want.abs() >= small) & (want.abs() <= f.max / 1.01)
    tol = want.abs() * (f32 + f.eps / 2 * 1.0001)
    assert int(ok.sum()) > n // 2 and ((y[:, 0].double() - want).abs() <= tol)[ok].all()


def test_a_recorded_call_has_a_gradient():
    """What the gradient's products could not take is refused when the call is recorded."""
    from resident_expert_routing_amd import binding as B
    from resident_expert_routing_amd import grouped, rows
    a = torch.ones(3, 1, dtype=BF16, device="cuda", requires_grad=True)
    b = torch.ones(1, (1 << 24) + 2, 1, dtype=BF16, device="cuda")
    offsets = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    with torch.no_grad():
        assert grouped.matmul(a, b, offsets, swiglu=True).shape == (3, (1 << 23) + 1)
    with pytest.raises(B.MoeError):
        grouped.matmul(a, b, offsets, swiglu=True)
    k = B.MOE_MAX_K + 1                     # more picks than a token's sum takes
    perm = torch.arange(3 * k, dtype=torch.int32, device="cuda")
    order = rows.RowOrder(perm, 3, k, perm.view(3, k))
    offsets[1] = 3 * k
    with torch.no_grad():
        assert grouped.matmul(a, b[:, :8], offsets, order=order).shape == (3 * k, 8)
    with pytest.raises(B.MoeError):
        grouped.matmul(a, b[:, :8], offsets, order=order)
    leaf = b[:, :8].clone().requires_grad_()
    y = grouped.matmul(a.detach(), leaf, offsets, order=order)
    assert (torch.autograd.grad(y, leaf, torch.ones_like(y))[0] == 3 * k).all()


@pytest.mark.parametrize("swiglu", [False, True])
def test_what_a_gradient_does_not_read_may_change(swiglu):
    """Rows may be written over where only their own gradient is wanted, and matrices likewise;
    what the wanted gradient reads is refused."""
    from resident_expert_routing_amd import grouped
    a, b, offsets, d = case([10, 0, 25], 24, 16, FP32, swiglu=swiglu)
    b1 = b.clone().requires_grad_()
    want = torch.autograd.grad(grouped.matmul(a.requires_grad_(), b1, offsets, swiglu=swiglu), [a, b1], d)
    a = a.detach()
    x, w = a.clone().requires_grad_(), b.clone()
    inner = x * 1
    y = grouped.matmul(inner, w, offsets, swiglu=swiglu)
    inner.add_(1)
    assert torch.equal(torch.autograd.grad(y, x, d)[0], want[0])
    y = grouped.matmul(x * 1, w, offsets, swiglu=swiglu)
    w.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        torch.autograd.grad(y, x, d)
    x, w = a.clone(), b.clone().requires_grad_()
    y = grouped.matmul(x, w, offsets, swiglu=swiglu)
    with torch.no_grad():
        w.add_(1)
    assert torch.equal(torch.autograd.grad(y, w, d)[0], want[1])
    y = grouped.matmul(x, w, offsets, swiglu=swiglu)
    x.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        torch.autograd.grad(y, w, d)


def test_hooks_see_all_that_is_kept():
    """Everything that a recorded call keeps for its gradient passes through torch's hooks for
    saved tensors, the order too, and may come back from elsewhere."""
    from resident_expert_routing_amd import grouped, rows
    gen = torch.Generator().manual_seed(8)
    T, k = 50, 2
    perm, offsets = (t.cuda() for t in bucketing([30, 50, 20], gen))
    a = torch.randn(T, 32, generator=gen).to(BF16).cuda().requires_grad_()
    b = torch.randn(3, 16, 32, generator=gen).to(BF16).cuda().requires_grad_()
    d = torch.randn(T * k, 16, generator=gen).to(BF16).cuda()
    order = rows.RowOrder(perm, T, k)
    seen = []
    def pack(t):
        seen.append(t.data_ptr())
        return t.cpu()
    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t.cuda()):
        y = grouped.matmul(a, b, offsets, order=order)
    assert {t.data_ptr() for t in (a, b, order.pos, order.perm)} <= set(seen)
    want = torch.autograd.grad(grouped.matmul(a, b, offsets, order=order), [a, b], d)
    for g, w in zip(torch.autograd.grad(y, [a, b], d), want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("swiglu,across", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("dtype,counts,N,K", [
    (BF16, [9, 0, 11], 24, 40),                                   # the streaming form, or small tiles
    (FP16, [70, 3, 67], 72, 136), (FP32, [70, 3, 67], 41, 35),    # small tiles
    (BF16, [300, 4, 90, 1, 129] * 20, 300, 72)])                  # large tiles
def test_an_assignment_named_twice(counts, N, K, swiglu, across, dtype):
    """As in dispatch: the earlier row of an assignment that the order names twice is zero, and
    has no part in a gradient."""
    from resident_expert_routing_amd import grouped, rows
    k, G = 2, len(counts)
    gen = torch.Generator().manual_seed(9)
    perm, offsets = bucketing(counts, gen, tail=sum(counts) % 2)
    M = perm.numel()
    early = torch.arange(0, M // 2, 3)
    perm[early] = perm[M // 2 + early // 2]
    perm[M // 2 - 1] = M                                          # names nothing
    index = torch.where((perm < 0) | (perm >= M), -1, perm // k)
    holes = index.clone()
    holes[early] = -1
    a = torch.randn(M // k, K, generator=gen).to(dtype).cuda().requires_grad_()
    b = (torch.randn(G, 2 * N if swiglu else N, K, generator=gen) * K ** -0.5).to(dtype).cuda()
    if across:
        b = b.transpose(1, 2).contiguous().transpose(1, 2)
    b = b.detach().requires_grad_()
    d = torch.randn(M, N, generator=gen).to(dtype).cuda()
    perm, offsets, holes = perm.cuda(), offsets.cuda(), holes.cuda()
    ref = Reference(a.detach(), b.detach(), offsets, holes, M, swiglu, dtype, d, token_sum=True)
    order = rows.RowOrder(perm, M // k, k)
    y = grouped.matmul(a, b, offsets, order=order, swiglu=swiglu)
    assert within(y.detach(), ref.out, ref.out_tol) and not y[holes < 0].any()
    with torch.no_grad():
        assert torch.equal(grouped.matmul(a, b, offsets, order=order, swiglu=swiglu), y)
    d[holes < 0] = float("nan")
    da, db = torch.autograd.grad(y, [a, b], d)
    assert within(da, ref.da, ref.da_tol)
    assert within(db, ref.db, ref.db_tol)
