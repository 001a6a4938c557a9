"""4-bit products at the edges: every form of the kernel, padding, layouts, values that are
no numbers, sizes past 32 bits, graphs and streams, refusals, and the layer."""
import pytest
import torch
from torch.autograd import forward_ad

from grouped_oracle import bucketing, within
from test_gpu_int4 import random_weight, reference, values

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def made(G, N, K, group=64, zeros=True, scale_dtype=BF16, seed=0):
    from resident_expert_routing_amd import int4
    gen = torch.Generator().manual_seed(seed)
    codes, scale, zero = random_weight((G,) if G else (), N, K, group, zeros, scale_dtype, gen)
    return int4.pack(codes, scale, zero, group=group), values(codes, scale, zero, group), gen


def spans(offsets):
    e = offsets.tolist()
    return [(g, lo, hi) for g, (lo, hi) in enumerate(zip(e, e[1:])) if hi > lo]


def form(M, N, G, swiglu):
    """The form that the kernel's launcher takes, by the rule in its comment."""
    per = lambda cols: -(-N // (cols // 2 if swiglu else cols))
    groups = min(G, M) if G else 1
    items = M // 16 + (groups if G else 1)
    thin = M <= 16 or M < 24 * groups
    if not thin and groups * per(256) >= 256:
        return "wide"
    if items * per(32) <= 256:
        return "few"
    return "mid" if items * per(128) < 640 else "thin"


# rows of the groups, N, the form
FORMS = [([1, 0, 3], 64, "few"), ([2] * 9, 1024, "mid"), ([1, 0, 2] * 120, 300, "thin"),
         ([9, 40, 3, 0] * 16, 1030, "thin"), ([70, 31, 0, 65, 1] * 65, 257, "wide")]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("group,swiglu,K", [(128, False, 384), (64, True, 200), (32, False, 650)])
@pytest.mark.parametrize("at", range(len(FORMS)))
def test_forms(at, group, swiglu, K, dtype):
    from resident_expert_routing_amd import int4
    counts, N, want = FORMS[at]
    N = N // 2 + 7 if swiglu else N
    w, (exact, sc), gen = made(len(counts), 2 * N if swiglu else N, K, group, zeros=group != 128,
                               seed=at)
    perm, offsets = bucketing(counts, gen, tail=3)
    M = perm.numel()
    taken = form(M, N, len(counts), swiglu)
    print(f"{M} rows, N {N}: {taken}", flush=True)
    assert taken == want or swiglu
    perm, offsets = perm.cuda(), offsets.cuda()
    a = torch.randn(M, K, generator=gen).to(dtype).cuda()
    out = torch.full((M, N), 5.0, dtype=dtype, device="cuda")
    int4.matmul(a, w, offsets=offsets, index=perm, swiglu=swiglu, out=out)
    for g, lo, hi in spans(offsets):
        y, tol = reference(a[perm[lo:hi].long()], exact[g], sc[g], swiglu, dtype)
        assert within(out[lo:hi], y, tol)
    assert (out[int(offsets[-1]):] == 5).all()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(17, 33), (40, 130), (5, 300)])
def test_padding_may_hold_anything(N, K, group):
    from resident_expert_routing_amd import int4
    w, _, gen = made(2, N, K, group)
    a = torch.randn(7, K, generator=gen).to(BF16).cuda()
    offsets = torch.tensor([0, 3, 7], dtype=torch.int32, device="cuda")
    want = int4.matmul(a, w, offsets=offsets)
    Np, Kp = w.codes.shape[1] * 16, w.codes.shape[2] * 128
    row = torch.arange(Np, device="cuda").view(-1, 1, 16, 1).expand(w.codes.shape[1:]) >= N
    # byte b of a word holds weights 2 b' and 2 b' + 1 of one parity; words behind K hold none
    word = torch.arange(64, device="cuda") // 4 * 8
    behind = (torch.arange(Kp // 128, device="cuda").view(-1, 1, 1) * 128 + word) >= K
    w.codes[:, row | behind] = 0xFF
    live = torch.zeros(Np, Kp // group, dtype=torch.bool, device="cuda")
    live[:N, :-(-K // group)] = True
    live = live.view(Np // 16, 16, -1).transpose(1, 2)
    w.scale[:, ~live] = float("nan")
    w.zero[:, ~live] = 0xFF
    assert torch.equal(int4.matmul(a, w, offsets=offsets), want)


def test_layouts():
    """Activations at odd addresses, an out among others, matrices at a distance, and types
    that differ."""
    from resident_expert_routing_amd import int4
    w, (exact, sc), gen = made(3, 48, 160)
    base = torch.randn(20, 200, generator=gen).to(BF16).cuda()
    a = base[:, 3:163]
    offsets = torch.tensor([0, 5, 5, 18], dtype=torch.int32, device="cuda")
    far = torch.zeros(3, 2 * w.codes[0].numel() + 16, dtype=torch.uint8, device="cuda")
    codes = far[:, :w.codes[0].numel()].view(w.codes.shape).copy_(w.codes)
    side = torch.zeros(3, w.scale[0].numel() + 4, dtype=w.scale.dtype, device="cuda")
    scale = side[:, :w.scale[0].numel()].view(w.scale.shape).copy_(w.scale)
    v = int4.Int4Weight(codes, scale, w.zero, N=48, K=160)
    for odt in (BF16, FP16, FP32):
        out = torch.full((22, 60), 2.0, dtype=odt, device="cuda")
        view = out[1:21, 5:53]
        assert int4.matmul(a, v, offsets=offsets, out=view) is view
        for g, lo, hi in spans(offsets):
            y, tol = reference(a[lo:hi], exact[g], sc[g], False, odt)
            assert within(view[lo:hi], y, tol)
        view[:18] = 2
        assert (out == 2).all()
        assert int4.matmul(a[:5], w[0], out_dtype=odt).dtype == odt
    t = torch.randn(160, 20, generator=gen).cuda()
    assert torch.equal(int4.matmul(t.t(), w[1]), int4.matmul(t.t().contiguous(), w[1]))
    one = torch.randn(1, 160, generator=gen).cuda().expand(20, 160)
    assert torch.equal(int4.matmul(one, w[1]), int4.matmul(one.contiguous(), w[1]))


def test_values_that_are_no_numbers():
    """A NaN in a row of a, or in a scale, stays in its row, or column."""
    from resident_expert_routing_amd import int4
    w, _, gen = made(0, 40, 256, zeros=False)
    a = torch.randn(9, 256, generator=gen).cuda()
    want = int4.matmul(a, w)
    bad = a.clone()
    bad[4, 77] = float("nan")
    got = int4.matmul(bad, w)
    keep = torch.arange(9, device="cuda") != 4
    assert torch.equal(got[keep], want[keep]) and got[4].isnan().all()
    w.scale[1, 2, 3] = float("nan")  # row 19
    got = int4.matmul(a, w)
    cols = torch.arange(40, device="cuda") != 19
    assert torch.equal(got[:, cols], want[:, cols]) and got[:, 19].isnan().all()
    x = torch.ones(20, 200, device="cuda")
    x[3, 150], x[7, 5], x[9, :64] = float("inf"), float("nan"), 0
    q = int4.quantize(x, 64)
    d = q.dequantize()
    assert d[3, 128:192].isnan().all() and d[7, :64].isnan().all() and not d[9, :64].any()
    ok = torch.ones(20, 200, dtype=torch.bool, device="cuda")
    ok[3, 128:192] = ok[7, :64] = False
    assert torch.isfinite(d[ok]).all()
    big = int4.quantize(torch.full((1, 32), 1e6, device="cuda"), 32, scale_dtype=FP16)
    assert big.scale[0, 0, 0].isnan()                      # past the scale's type


def test_sizes_past_32_bits():
    from resident_expert_routing_amd import int4
    G, N, K = 300, 4096, 4096
    w = int4.Int4Weight.empty(G, N, K, zeros=True)
    assert w.codes.numel() > 2 ** 31
    small, (exact, sc), gen = made(0, N, K, 128)
    w.codes[-1], w.scale[-1], w.zero[-1] = small.codes, small.scale, small.zero
    a = torch.randn(20, K, generator=gen).to(BF16).cuda()
    offsets = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = 20
    y, tol = reference(a, exact, sc, False, BF16)
    assert within(int4.matmul(a, w, offsets=offsets), y, tol)


@pytest.mark.parametrize("G", [257, 3000])
def test_many_groups(G):
    from resident_expert_routing_amd import int4
    w, (exact, sc), gen = made(G, 20, 64, 32)
    counts = ((torch.rand(G, generator=gen) < 0.05).int() * 3).tolist()
    counts[-1] = 20
    perm, offsets = bucketing(counts, gen)
    offsets = offsets.cuda()
    a = torch.randn(perm.numel(), 64, generator=gen).to(BF16).cuda()
    got = int4.matmul(a, w, offsets=offsets)
    for g, lo, hi in spans(offsets):
        y, tol = reference(a[lo:hi], exact[g], sc[g], False, BF16)
        assert within(got[lo:hi], y, tol)


def test_refusals():
    from resident_expert_routing_amd import int4
    w, _, gen = made(2, 32, 128)
    a = torch.randn(6, 128, generator=gen).to(BF16).cuda()
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    ok = dict(a=a, w=w, offsets=off)
    int4.matmul(**ok)
    for kw in (dict(a=a.int()), dict(a=a[:, :64]), dict(a=a.cpu()), dict(offsets=off.long()),
               dict(offsets=off[:2]), dict(offsets=None), dict(w=w[0]), dict(index=off.long()),
               dict(out=torch.empty(6, 31, device="cuda")), dict(out_dtype=torch.int8),
               dict(out=torch.empty(32, 6, device="cuda").t()),
               dict(out=torch.empty(6, 32, device="cuda", requires_grad=True)),
               dict(a=a.clone().requires_grad_())):
        with pytest.raises(ValueError):
            int4.matmul(**(ok | kw))
    with pytest.raises(RuntimeError, match="moe_int4_matmul"):
        int4.matmul(**ok, index=torch.zeros(3, dtype=torch.int32, device="cuda"), index_div=0)
    with pytest.raises(ValueError, match="even"):
        int4.matmul(a, made(0, 33, 128)[0], swiglu=True)
    with forward_ad.dual_level(), pytest.raises(ValueError, match="tangent"):
        int4.matmul(forward_ad.make_dual(a, a), w, offsets=off)
    c, s, z = w.codes, w.scale, w.zero
    for args, kw in (((c.int(), s, z), {}), ((c, s.float(), z), {}), ((c, s, z.int()), {}),
                     ((c, s[:, :, :1], z), {}), ((c, s, z[:1]), {}), ((c.cpu(), s, z), {}),
                     ((c, s, z), dict(N=49)), ((c, s, z), dict(K=200)), ((c, s, z), dict(N=0)),
                     ((c[:, :, :, ::2], s, z), {}), ((c.transpose(-1, -2), s, z), {})):
        with pytest.raises(ValueError):
            int4.Int4Weight(*args, **(dict(N=32, K=128) | kw))
    for bad in (dict(group=48), dict(scale_dtype=FP32)):
        with pytest.raises(ValueError):
            int4.quantize(a, **bad)
    with pytest.raises(ValueError):
        int4.quantize(a.clone().requires_grad_())
    with pytest.raises(ValueError):
        w.load(a)                                       # several matrices
    with pytest.raises(ValueError):
        w[0].load(a[:, :64])
    with pytest.raises(ValueError):
        w[0].load(a, 8)                                 # inside a tile
    with pytest.raises(ValueError):
        int4.Int4Experts(w, w)


def test_captured_and_replayed():
    from resident_expert_routing_amd import int4
    w, _, gen = made(4, 96, 256, 128, zeros=False)
    a = torch.randn(12, 256, generator=gen).to(BF16).cuda()
    orders = [[t.cuda() for t in bucketing(c, gen, tail=24 - sum(c))]
              for c in ([1, 0, 20, 3], [6] * 4, [0, 0, 0, 2])]
    perm, offsets = orders[0][0].clone(), orders[0][1].clone()
    out = torch.zeros(24, 48, dtype=BF16, device="cuda")
    call = lambda to: int4.matmul(a, w, offsets=offsets, index=perm, index_div=2, swiglu=True, out=to)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for p, o in orders:
        perm.copy_(p), offsets.copy_(o), a.mul_(1.25), out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, call(torch.zeros_like(out)))


def test_two_streams():
    from resident_expert_routing_amd import int4
    sets = [made(0, 512, 1024, 128, seed=s)[0] for s in range(2)]
    a = torch.randn(5, 1024, device="cuda").to(FP16)
    want = [int4.matmul(a, w) for w in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(int4.matmul(a, sets[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])


@pytest.mark.parametrize("T,H,E,k,I,S,resident,zeros", [
    (1, 256, 16, 4, 128, 10, 10, False), (8, 512, 64, 8, 256, 40, 40, True),
    (9, 256, 16, 4, 96, 10, 3, False), (70, 320, 8, 2, 160, 8, 8, True)])
def test_layer(T, H, E, k, I, S, resident, zeros):
    """Routing, 4-bit experts and combine against the same chain in float64 with the weights
    as they are stored.  h, the rows and the sum are each rounded to bf16, at most 2^-9 of a
    value: relative L2 within 3 * 2^-9."""
    from test_gpu_int8 import routed
    from resident_expert_routing_amd import int4
    from resident_expert_routing_amd import runtime as R
    buf, x, (wg, wu, wd), args = routed(T, H, E, k, I, S, resident, T)
    ex = int4.Int4Experts.from_weights(wg, wu, wd, group=32, zeros=zeros)
    out = ex.forward(x, buf.slot_offsets, buf.perm, buf.sel_weight)
    gu, dn = ex.gate_up.dequantize().double(), ex.down.dequantize().double()
    # what is stored is the weights to half a step of their group: scales are at most a
    # seventh (a fifteenth of twice that) of the largest weight, rounded by 2^-9
    assert float((gu[:, :I] - wg.double()).abs().max()) <= float(wg.abs().max()) / 7 * 0.51 + 1e-6 \
        or zeros
    off, perm = buf.slot_offsets.tolist(), buf.perm.long()
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for s in range(S):
        p = perm[off[s]:off[s + 1]]
        if p.numel():
            z = x[p // k].double() @ gu[s].t().contiguous()
            h = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
            want.index_add_(0, p // k, (h @ dn[s].t().contiguous())
                            * buf.sel_weight.view(-1)[p, None].double())
    rel = float((out.double() - want).norm() / want.norm())
    print(f"relative L2 {rel:.2e}", flush=True)
    assert rel <= 3 * 2.0 ** -9
    hist = torch.zeros(E, dtype=torch.float64, device="cuda")
    step = R.layer_step_int4(buf, x, args[0], None, args[1], hist, ex)
    assert torch.equal(step, out) and float(hist.sum()) > 0
    other = int4.Int4Experts.empty(S + 1, H, I, "cuda")
    for wrong, e in ((x[:, :-1], ex), (x.float(), ex), (x, other), (torch.cat([x, x]), ex)):
        before = hist.clone()
        with pytest.raises(ValueError):
            R.layer_step_int4(buf, wrong, args[0], None, args[1], hist, e)
        assert torch.equal(hist, before)


def test_up_rows_inside_a_tile():
    """Experts whose gate rows end inside a tile of sixteen: loaded and multiplied alike."""
    from resident_expert_routing_amd import int4
    S, H, I = 3, 100, 21
    gen = torch.Generator().manual_seed(2)
    gate, up = (torch.randn(S, I, H, generator=gen).to(BF16).cuda() for _ in range(2))
    down = torch.randn(S, H, I, generator=gen).to(BF16).cuda()
    ex = int4.Int4Experts.from_weights(gate, up, down, group=32, zeros=True)
    whole = int4.quantize(torch.cat([gate, up], 1), 32, zeros=True)
    assert torch.equal(ex.gate_up.dequantize(), whole.dequantize())
    x = torch.randn(6, H, generator=gen).to(BF16).cuda()
    offsets = torch.tensor([0, 2, 2, 6], dtype=torch.int32, device="cuda")
    perm = torch.randperm(6, generator=gen).int().cuda()
    got = int4.matmul(x, ex.gate_up, offsets=offsets, index=perm, swiglu=True)
    w = whole.dequantize().double()
    sc = torch.full_like(w, float(whole.scale.float().max()))
    for g, lo, hi in spans(offsets):
        y, tol = reference(x[perm[lo:hi].long()], w[g], sc[g], True, BF16)
        assert within(got[lo:hi], y, tol)
    rows = ex.rows(x, offsets, perm, 1)
    assert rows.shape == (6, H) and torch.isfinite(rows).all()


def test_scales_that_are_no_groups():
    from resident_expert_routing_amd import int4
    w, _, _ = made(0, 32, 128, zeros=False)
    for n in (0, 3, 8):
        with pytest.raises(ValueError):
            int4.Int4Weight(w.codes, torch.empty(2, n, 16, dtype=BF16, device="cuda"), N=32, K=128)


def test_pack_has_no_gradient():
    """Scales that want a gradient, or carry a tangent, are refused; under no_grad they pass."""
    from resident_expert_routing_amd import int4
    codes = torch.randint(0, 16, (16, 128), dtype=torch.uint8, device="cuda")
    scale = torch.rand(16, 2, device="cuda").to(BF16).requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        int4.pack(codes, scale, group=64)
    with torch.no_grad():
        assert not int4.pack(codes, scale, group=64).scale.requires_grad
    with forward_ad.dual_level(), pytest.raises(ValueError, match="tangent"):
        int4.pack(codes, forward_ad.make_dual(scale.detach(), scale.detach()), group=64)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize_of_the_largest_numbers(group, dtype):
    """Weights whose range float32 does not hold, but whose scale its type does."""
    from resident_expert_routing_amd import int4
    gen = torch.Generator().manual_seed(6)
    w = ((torch.rand(20, 256, generator=gen) * 2 - 1) * torch.finfo(dtype).max).to(dtype).cuda()
    for zeros in (False, True):
        q = int4.quantize(w, group, zeros=zeros)
        v = w.double().view(20, -1, group)
        lo, hi = v.amin(2), v.amax(2)
        assert (hi - lo).max() > torch.finfo(FP32).max
        want = (hi - lo) / 15 if zeros else torch.maximum(hi, -lo) / 7
        scale = q.scale.double().transpose(1, 2).reshape(-1, q.scale.shape[1])[:20]
        assert ((scale - want).abs() <= want * (2.0 ** -8 + 2.0 ** -22)).all()
        # half a step, and with a zero point its own rounding and the scale's of 15 steps
        step = scale.unsqueeze(2) * ((1 + 15 * 2.0 ** -8 if zeros else 0.5 + 8 * 2.0 ** -8) + 1e-5)
        # steps times scale in float64: seven steps of a scale that was rounded up may pass
        # float32's largest number by that rounding, 2^-8
        steps = int4.Int4Weight(q.codes, torch.ones_like(q.scale), q.zero, N=20, K=256).dequantize()
        got = steps.double().view(20, -1, group) * scale.unsqueeze(2)
        assert ((got - v).abs() <= step).all()


def agree(got, want, tol):
    """Where want is a number, within tol; the same infinities and NaN elsewhere."""
    fine = torch.isfinite(want)
    got = got.double()
    assert torch.equal(fine, torch.isfinite(got))
    assert torch.equal(want.isnan(), got.isnan())
    inf = ~fine & ~want.isnan()
    assert torch.equal(want[inf], got[inf])
    worst = ((got - want).abs() / tol.clamp_min(1e-300))[fine]
    assert worst.numel() == 0 or float(worst.max()) <= 1, float(worst.max())


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("group,zeros,swiglu,K", [(128, False, False, 384), (64, True, False, 200),
                                                  (32, True, True, 650)])
@pytest.mark.parametrize("at", range(len(FORMS)))
def test_infinities(at, group, zeros, swiglu, K, dtype):
    """An infinite activation gives the definition's infinities, and NaN only where the weight is
    zero or another infinity meets it; other rows' results do not change by a bit."""
    from resident_expert_routing_amd import int4
    counts, N, _ = FORMS[at]
    N = N // 2 + 7 if swiglu else N
    w, (exact, sc), gen = made(len(counts), 2 * N if swiglu else N, K, group, zeros, seed=at)
    perm, offsets = bucketing(counts, gen)
    M = perm.numel()
    a = torch.randn(M, K, generator=gen).to(dtype)
    bad = a.clone()
    inf = float("inf")
    rows = torch.randperm(M, generator=gen)[:max(1, M // 3)]
    for i, r in enumerate(rows.tolist()):
        at_k = torch.randint(0, K, (2,), generator=gen)
        for n, v in ((0, (inf, -inf, inf, float("nan"))[i % 4]),
                     (1, (a[r, at_k[1]], a[r, at_k[1]], -inf, 1.0)[i % 4])):
            bad[r, at_k[n]] = v
    perm, offsets = perm.cuda(), offsets.cuda()
    call = lambda x: int4.matmul(x.cuda(), w, offsets=offsets, index=perm, swiglu=swiglu,
                                 out_dtype=FP32)
    got, clean = call(bad), call(a)
    touched = torch.zeros(M, dtype=torch.bool)
    touched[rows] = True
    same = ~touched.cuda()[perm.long()]
    assert torch.equal(got[same], clean[same])
    x = bad.cuda().double()
    for g, lo, hi in spans(offsets):
        xs = x[perm[lo:hi].long()]
        # products one by one: a library's may meet an infinity with a zero of its own
        y = torch.stack([(r * exact[g]).sum(1) for r in xs])
        e = 2 * (K + 16) * 2.0 ** -23 * torch.stack(
            [(r.abs().nan_to_num(0, 0, 0) * 31 * sc[g]).sum(1) for r in xs])
        if swiglu:
            gt, up, eg, eu = y[:, :N], y[:, N:], e[:, :N], e[:, N:]
            y = gt / (1 + torch.exp(-gt)) * up
            low = gt == -inf                        # -inf * 0
            y = torch.where(low, torch.full_like(y, float("nan")), y)
            s = torch.sigmoid(gt)
            e = 1.1 * eg * (up.abs() + eu) + (gt * s).abs() * eu + \
                (1.25 * gt.abs() + 12) * 2.0 ** -24 * y.abs()
            e = e.nan_to_num(0, 0, 0)
        agree(got[lo:hi], y, e + 2.0 ** -24 * y.abs().nan_to_num(0, 0, 0) + 1e-30)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("group,zeros", [(128, False), (64, True), (32, False)])
def test_large_and_small_activations(group, zeros, dtype):
    """Up to the type's largest number and down to 2^-100, against weights of -1, 0 and 1 steps:
    sums that float32 holds are right."""
    from resident_expert_routing_amd import int4
    gen = torch.Generator().manual_seed(3)
    N, K, rows = 40, 300, 24
    n = -(-K // group)
    zero = torch.randint(1, 15, (N, n), dtype=torch.uint8, generator=gen)
    base = zero.repeat_interleave(group, 1)[:, :K] if zeros else torch.full((N, K), 8, dtype=torch.uint8)
    codes = (base.int() + torch.randint(-1, 2, (N, K), generator=gen)).to(torch.uint8).cuda()
    scale = (torch.rand(N, n, generator=gen) + 0.5).mul(2.0 ** -10).to(BF16).cuda()
    zero = zero.cuda() if zeros else None
    w = int4.pack(codes, scale, zero, group=group)
    exact, sc = values(codes, scale, zero, group)
    big = torch.finfo(dtype).max
    a = torch.randn(rows, K, generator=gen).clamp(-4, 4)
    for r in range(rows):
        if r < 8:                       # one of the largest among ordinary ones
            a[r, 11 * r + 5] = big * (-1) ** r
        elif r < 16:                    # all large: sums of at most 128 of them
            a[r] *= 2.0 ** (117 + (r - 8) // 2 % 2)
        else:
            a[r] *= 2.0 ** -100
    a = a.to(dtype).cuda()
    got = int4.matmul(a, w, out_dtype=FP32)
    want = a.double() @ exact.t().contiguous()
    tol = (K + 16) * 2.0 ** -22 * (a.double().abs() @ sc.t().contiguous()) * (
        torch.ones(rows, 1, dtype=torch.float64, device="cuda"))
    tol[16:] *= 31                      # 16-bit activations there: of a (16 + code), corrected
    tol[:16] += 2.0 ** -20 * want[:16].abs()
    assert torch.isfinite(want.float()).all()
    agree(got, want, tol + 2.0 ** -133)
