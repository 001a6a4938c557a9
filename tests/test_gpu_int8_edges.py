"""8-bit products and experts at the edges: saturating gates, tiles mapped to the
XCDs in blocks, batches that do not fit."""
import numpy as np
import pytest
import torch

from gpu_helpers import say

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
UNDER = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import resident_expert_routing_amd  # noqa: F401
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def tiles_of(M, N, swiglu, G=0):
    """(tiled form?, items x columns of 64-row tiles) by the rule of few_tiles."""
    cols = -(-N // (128 if swiglu else 256))
    items, thin = -(-M // 64), False
    if G:
        groups = min(G, M)
        items, thin = max(items, groups), M < 4 * groups
    return items * cols >= (192 if thin else 48), items * cols


@pytest.mark.parametrize("N", [40, 1801])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_saturating_gates(N, dtype):
    """SwiGLU with gates over +-127 and beyond, in the streaming and the tiled form.

    Gate and up values are exact: one product each of small integers and scales
    that are powers of two.  So the only errors are the epilogue's: for |g| <= 64
    the argument of exp, its instruction (2 units of 2^-24 after the argument's
    1.25 |g|), a sum (1), a reciprocal (2) and two products (2); below -64 two
    halves of the argument's 1.25 |g|, two exponentials (4) and three products (3);
    above, less.  (1.25 |g| + 8) * 2^-24 of the value holds all, then the rounding
    to the type.  Largest magnitudes of the exact values, 127 * 127 * 2^20 * 16, are
    finite in float32 and overflow in fp16, as they should."""
    from resident_expert_routing_amd import int8
    tiled, n = tiles_of(255, N, True)
    say(f"gates N={N} {dtype} tiled={tiled} ({n} tiles)")
    assert tiled == (N > 100)
    M, K = 255, 16
    a = torch.zeros(M, K, dtype=torch.int8)
    a[:, 0] = torch.arange(-127, 128)             # the gate's factor
    a[:, 1] = torch.arange(M) % 13 - 6            # the up's
    b = torch.zeros(2 * N, K, dtype=torch.int8)
    b[:N, 0] = torch.arange(N) % 16 + 1           # gates: r * (1 .. 16) / 16 and / 8
    b[N:, 1] = torch.arange(N) % 127 + 1
    sb = torch.ones(2 * N)
    sb[:N] = torch.where(torch.arange(N) % 3 == 0, 0.125, 0.0625)
    sb[N:] = 2.0 ** (20 - torch.arange(N) % 21).double()
    got = int8.matmul(a.cuda(), torch.ones(M, device="cuda"), b.cuda(), sb.cuda(), swiglu=True,
                      out_dtype=dtype).cpu().double()
    z = (a.double() @ b.double().t()) * sb.double()
    g, u = z[:, :N], z[:, N:]
    assert float(g.min()) < -200 and float(g.max()) > 200
    want = g / (1 + torch.exp(-g)) * u
    most = torch.finfo(dtype).max
    eps = torch.finfo(dtype).eps / 2
    bound = (1.25 * g.abs() + 8) * 2.0 ** -24 * want.abs() * (1 + eps) + eps * want.abs() \
        + UNDER[dtype]
    bound = torch.where(g < -174, bound + want.abs(), bound)   # h is below every normal number
    fits = want.abs() < most * (1 - 4 * eps)
    off = (got - want).abs()
    assert bool((off[fits] <= bound[fits]).all()), float((off / bound)[fits].max())
    over = want.abs() > most * (1 + 4 * eps)
    assert bool(torch.isinf(got[over]).all())
    assert not bool(torch.isnan(got).any())
    # values that are normal numbers of the type are not lost
    normal = (g > -174) & (want.abs() > 2 * torch.finfo(dtype).tiny)
    assert bool((got[normal] != 0).all())


def test_gates_that_are_no_numbers():
    """Infinite and NaN scales reach only the rows they belong to; silu(-inf) is
    NaN, as g / (1 + exp(-g)) is."""
    from resident_expert_routing_amd import int8
    for N in (40, 1801):
        M, K = 255, 16
        a, b = torch.ones(M, K, dtype=torch.int8), torch.ones(2 * N, K, dtype=torch.int8)
        sa = torch.full((M,), 0.125)
        sa[3], sa[7] = float("nan"), float("inf")
        b[1] = -1
        y = int8.matmul(a.cuda(), sa.cuda(), b.cuda(), torch.ones(2 * N, device="cuda"),
                        swiglu=True, out_dtype=torch.float32).cpu()
        assert torch.isnan(y[3]).all()
        assert torch.isnan(y[7, 1]) and bool((y[7, 2:] == float("inf")).all())
        rest = torch.ones(M, dtype=torch.bool)
        rest[[3, 7]] = False
        assert bool(torch.isfinite(y[rest]).all())


def test_batches_that_do_not_fit_are_refused():
    """Token rows, perm or buffers that do not belong together, rows that the
    router would read as something else: refused, and the demand is not counted."""
    from resident_expert_routing_amd import int8
    from resident_expert_routing_amd import runtime as R
    T, H, E, k, I, S = 12, 256, 16, 4, 128, 10
    dev = torch.device("cuda", 0)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    w_router = (torch.randn(E, H, generator=g) / 16).cuda()
    slot = torch.full((E,), -1, dtype=torch.int32)
    slot[:S] = torch.arange(S, dtype=torch.int32)
    slot = slot.cuda()
    buf = R.LayerBuffers(T, H, E, k, I, S, dev)
    hist = torch.zeros(E, dtype=torch.float64, device="cuda")
    w = [(torch.randn(S, *s, generator=g) / 16).cuda() for s in ((I, H), (I, H), (H, I))]
    ex = int8.Int8Experts.from_weights(*w)

    def step(x, ex=ex):
        return R.layer_step_int8(buf, x, w_router, None, slot, hist, ex)

    want = step(x)
    counted = hist.clone()
    assert float(counted.sum()) > 0
    wide = torch.zeros(T, 2 * H, dtype=torch.bfloat16, device="cuda")
    wide[:, ::2] = x
    for bad in (x.view(torch.int16), x.half(), x.float(), x[:-1], x[:, :-8].contiguous(),
                wide[:, ::2], wide[:, :H], x.cpu(), x.clone().requires_grad_()):
        with pytest.raises(ValueError):
            step(bad)
    for kw in (dict(row_dtype=torch.float64), dict(inner_dtype=torch.int8)):
        with pytest.raises(ValueError, match="rows are"):
            R.layer_step_int8(buf, x, w_router, None, slot, hist, ex, **kw)
    for s in (S - 1, S + 1):
        with pytest.raises(ValueError, match="slots"):
            step(x, int8.Int8Experts.empty(s, H, I, dev))
    with pytest.raises(ValueError):
        step(x, int8.Int8Experts.empty(S, 2 * H, I, dev))
    torch.cuda.synchronize()
    assert torch.equal(hist, counted)
    args = (buf.slot_offsets, buf.perm)
    fine = dict(row_dtype=torch.float32, inner_dtype=torch.float32)
    assert torch.equal(R.layer_step_int8(buf, x, w_router, None, slot, hist, ex, **fine),
                       ex.forward(x, *args, buf.sel_weight, **fine))
    for bad in (x[:-1], torch.cat((x, x)), x.view(torch.int16), x.double(), x[0]):
        with pytest.raises(ValueError):
            ex.forward(bad, *args, buf.sel_weight)
    with pytest.raises(ValueError, match="perm"):
        ex.rows(x[:-1], *args, k)
    with pytest.raises(ValueError, match="perm"):
        ex.rows(x, *args, k - 1)
    assert torch.equal(ex.forward(x, *args, buf.sel_weight), want)
    m = int(buf.slot_offsets[-1])                 # the rows that are in a slot, and no others
    assert torch.equal(ex.rows(x, args[0], args[1][:m], k), ex.rows(x, *args, k)[:m])
    # a matrix of other strides is taken where the router is not asked
    assert torch.equal(ex.forward(wide[:, ::2], *args, buf.sel_weight), want)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T", [3, 70])
def test_types_between_the_products_are_the_callers(T, dtype):
    """inner_dtype and row_dtype: the same chain call by call, and the weighted sum
    of float32 rows within its own roundings, (k + 1) * 2^-24 of the magnitudes and
    one to the type.  The defaults (bf16, x's type) are what they were."""
    from resident_expert_routing_amd import int8, rows
    H, k, I, S = 200, 3, 72, 6
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(dtype).cuda()
    sel = torch.stack([torch.randperm(S, generator=g)[:k] for _ in range(T)])
    perm = torch.sort(sel.reshape(-1), stable=True).indices.int().cuda()
    off = torch.zeros(S + 1, dtype=torch.int32)
    off[1:] = torch.bincount(sel.reshape(-1), minlength=S).cumsum(0)
    off = off.cuda()
    w = torch.rand(T, k, generator=g).cuda()
    ex = int8.Int8Experts.from_weights(*((torch.randn(S, *s, generator=g) / s[1] ** 0.5).cuda()
                                         for s in ((I, H), (I, H), (H, I))))
    order = rows.RowOrder(perm, T, k)
    q, s = int8.quantize(x)

    def chain(inner, row):
        h = int8.matmul(q, s, ex.gate_up, ex.gate_up_scale, offsets=off, index=perm, index_div=k,
                        swiglu=True, out_dtype=inner)
        return int8.matmul(*int8.quantize(h), ex.down, ex.down_scale, offsets=off, out_dtype=row)

    bf16, f32 = torch.bfloat16, torch.float32
    assert torch.equal(ex.rows(x, off, perm, k), chain(bf16, f32))
    assert torch.equal(ex.forward(x, off, perm, w), rows.combine(chain(bf16, dtype), order, w))
    y = chain(f32, f32)
    assert torch.equal(ex.rows(x, off, perm, k, inner_dtype=f32), y)
    assert not torch.equal(y, chain(bf16, f32))
    out = ex.forward(x, off, perm, w, row_dtype=f32, inner_dtype=f32)
    assert out.dtype == dtype
    terms = y.cpu().double()[order.pos.cpu().long()] * w.cpu().double().unsqueeze(2)
    want, mag = terms.sum(1), terms.abs().sum(1)
    eps = torch.finfo(dtype).eps / 2
    bound = (k + 1) * 2.0 ** -24 * mag * (1 + eps) + eps * want.abs() + UNDER[dtype]
    assert bool(((out.cpu().double() - want).abs() <= bound).all())
    with pytest.raises(ValueError):
        ex.forward(x, off, perm, w, row_dtype=torch.float64)
    with pytest.raises(ValueError):
        ex.forward(x, off, perm, w, inner_dtype=torch.int8)


def block_mapping(M, N, swiglu, G=0):
    """(tiles dealt to the XCDs in blocks?, items, columns), by the host's rule."""
    cols = -(-N // (128 if swiglu else 256))
    groups = min(G, M)
    if G and (M // 320 + groups) * cols >= 256:
        R = 320
    else:
        cost = {}
        for r in (320, 256, 192, 128, 64):
            items = M // r + groups if G else -(-M // r)
            cost[r] = -(-items * cols // 256) * (r + 256)
        R = min(cost, key=lambda r: (cost[r], -r))
    items = M // R + (groups if G else 1)
    return tiles_of(M, N, swiglu, G)[0] and M > 128 * max(G, 1) and items * cols >= 2048, items, cols


@pytest.mark.parametrize("M,N,sizes", [
    (5201, 33000, None),                                        # 17 items, 129 columns
    (5120, 32768, None),
    (2900, 60100, None),
    (3209, 33000, [700, 0, 321, 64, 900, 1, 640, 574]),         # 18 items
    (5127, 30000, [2500, 2618]),
    (4099, 24600, [129, 1000, 0, 65, 320, 1, 191, 639, 4, 300, 257, 700]),
])
@pytest.mark.parametrize("swiglu", [False, True])
def test_tiles_in_blocks(M, N, sizes, swiglu):
    """Products of many tiles deal them to the XCDs in blocks of 8 x 4: every tile
    is computed once, also at the ends of items and columns, and the rows behind the
    last group are left.  Sums are below 2^24, so float64 has them exactly."""
    from resident_expert_routing_amd import int8
    K = 64
    N = N // 2 if swiglu else N
    G = len(sizes) if sizes else 0
    in_blocks, items, cols = block_mapping(M, N, swiglu, G)
    say(f"blocks M={M} N={N} G={G} swiglu={swiglu}: {items} items x {cols} columns")
    assert in_blocks
    dtype = DTYPES[(M + swiglu) % 2]
    gen = torch.Generator(device="cuda").manual_seed(M)
    wide = 2 * N if swiglu else N
    lead = (G,) if G else ()
    a = torch.randint(-127, 128, (M, K), device="cuda", generator=gen, dtype=torch.int8)
    b = torch.randint(-127, 128, (*lead, wide, K), device="cuda", generator=gen, dtype=torch.int8)
    # y is up to 3, so that fp16 holds the products of gate and up
    sa = torch.rand(M, device="cuda", generator=gen) * 1e-3 + 1e-4
    sb = torch.rand(*lead, wide, device="cuda", generator=gen) * 1e-3 + 1e-4
    edges = np.concatenate([[0], np.cumsum(sizes)]) if G else np.array([0, M])
    off = torch.as_tensor(edges.astype(np.int32)).cuda() if G else None
    out = torch.full((M, N), 77.0, dtype=dtype, device="cuda")
    got = int8.matmul(a, sa, b, sb, offsets=off, swiglu=swiglu, out=out)
    eps = torch.finfo(dtype).eps / 2
    for g, (lo, hi) in enumerate(zip(edges, edges[1:])):
        bg, sg = (b[g], sb[g]) if G else (b, sb)
        for i in range(int(lo), int(hi), 1024):
            rows = slice(i, min(i + 1024, int(hi)))
            z = (a[rows].double() @ bg.double().t().contiguous()) * sa[rows].double()[:, None] * sg
            if swiglu:
                gate, up = z[:, :N], z[:, N:]
                si = gate / (1 + torch.exp(-gate))
                want = si * up
                err = 1.1 * 3 * 2.0 ** -24 * (gate * up).abs() + \
                    (1.5 * gate.abs() + 12) * 2.0 ** -24 * want.abs()
            else:
                want, err = z, 3.01 * 2.0 ** -24 * z.abs()
            bound = err * 1.01 + eps * (want.abs() + err) + UNDER[dtype]
            assert bool(((got[rows].double() - want).abs() <= bound).all()), (g, i)
    assert bool((got[int(edges[-1]):] == 77.0).all())


def small_layer(T, H=256, E=16, k=4, I=96, S=10, seed=1):
    """layer_step_int8's arguments for a layer of S resident experts."""
    from resident_expert_routing_amd import int8
    from resident_expert_routing_amd import runtime as R
    dev = torch.device("cuda", 0)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    w_router = (torch.randn(E, H, generator=g) / H ** 0.5).cuda()
    slot = torch.full((E,), -1, dtype=torch.int32)
    slot[torch.randperm(E, generator=g)[:S]] = torch.arange(S, dtype=torch.int32)
    w = [(torch.randn(S, *s, generator=g) / s[1] ** 0.5).cuda() for s in ((I, H), (I, H), (H, I))]
    hist = torch.zeros(E, dtype=torch.float64, device="cuda")
    return R.LayerBuffers(T, H, E, k, I, S, dev), x, w_router, None, slot.cuda(), hist, \
        int8.Int8Experts.from_weights(*w)


@pytest.mark.parametrize("T", [1, 33, 300])
def test_layer_step_captured_and_replayed(T):
    """The whole int8 layer step in a graph: every replay, with new rows and eager
    steps between, gives the eager result; so does a step on another stream."""
    from resident_expert_routing_amd import runtime as R
    buf, x, w_router, _, slot, hist, ex = small_layer(T)
    other = small_layer(T)[0]

    def inputs(seed):
        g = torch.Generator().manual_seed(seed)
        return torch.randn(T, x.shape[1], generator=g).to(torch.bfloat16).cuda()

    def eager(rows):
        return R.layer_step_int8(other, rows, w_router, None, slot, torch.zeros_like(hist), ex)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = R.layer_step_int8(buf, x, w_router, None, slot, hist, ex)
    side.synchronize()
    assert torch.equal(got, eager(x))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = R.layer_step_int8(buf, x, w_router, None, slot, hist, ex)
    for seed in (5, 6, 7, 5):
        rows = inputs(seed)
        x.copy_(rows)
        torch.cuda.synchronize()
        graph.replay()
        want = eager(rows)
        torch.cuda.synchronize()
        assert torch.equal(out, want), seed


def test_two_layers_at_once():
    """Two layers on two streams, several steps each: neither sees the other's."""
    from resident_expert_routing_amd import runtime as R
    layers = [small_layer(40, seed=1), small_layer(200, I=160, seed=2)]
    want = [R.layer_step_int8(*layer) for layer in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [[], []]
    for _ in range(6):
        for i, (layer, stream) in enumerate(zip(layers, streams)):
            with torch.cuda.stream(stream):
                got[i].append(R.layer_step_int8(*layer))
    torch.cuda.synchronize()
    for outs, ref in zip(got, want):
        assert all(torch.equal(o, ref) for o in outs)
