"""moe_positions, moe_dispatch, moe_combine and their gradients against the
formulas in float64 on the CPU.

Tolerances, per element: a value that the kernel computes with at most m float32
roundings of terms whose magnitudes sum to A, and then rounds once to the
element type, is within m * 2^-24 * A + eps/2 * |value| (+ half the type's
smallest subnormal) of the exact one; m = 1 for a scaled row, k + 1 for a sum of
k rows (one fused multiply-add each), and at most H + 12 for a dot product (no
term passes more than H sums, six steps of a wave and four waves)."""
import numpy as np
import pytest
import torch

from gpu_helpers import say

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# half of a type's smallest subnormal
UNDER = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import resident_expert_routing_amd  # noqa: F401
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def batch(T, k, S, seed, absent=0.0):
    """perm as moe_route writes it for random picks, some absent; float32 weights."""
    rng = np.random.default_rng(seed)
    sel = np.stack([rng.permutation(max(S, k))[:k] for _ in range(T)]) if T else \
        np.zeros((0, k), int)
    sel = np.where((sel >= S) | (rng.random(sel.shape) < absent), -1, sel)
    if absent and T > 1:
        sel[T // 2] = -1                       # a token without a single row
    flat = sel.reshape(-1)
    there = np.nonzero(flat >= 0)[0]
    order = there[np.argsort(flat[there], kind="stable")]
    perm = np.full(T * k, -1, np.int32)
    perm[:len(order)] = order
    w = rng.random((T, k)).astype(np.float32)
    return perm, w


def reference(perm, T, k):
    pos = np.full(T * k, -1, np.int64)
    there = np.nonzero((perm >= 0) & (perm < T * k))[0]
    pos[perm[there]] = there
    return pos.reshape(T, k)


def f64(t):
    return t.detach().cpu().double().numpy()


def close(got, want, mag, m, dtype, what):
    """|got - want| within the bound of the module's docstring."""
    got = f64(got)
    eps = 0.0 if dtype is None else torch.finfo(dtype).eps / 2
    under = 0.0 if dtype is None else UNDER[dtype]
    bound = m * 2.0 ** -24 * mag * (1 + eps) + eps * np.abs(want) + under
    off = np.abs(got - want)
    assert got.shape == want.shape
    assert np.all(off <= bound), (what, float(np.max(off - bound)), float(off.max()))


def spread_ref(x, perm, k, w):
    y = np.zeros((len(perm), x.shape[1]))
    there = np.nonzero(perm >= 0)[0]
    a = perm[there]
    y[there] = x[a // k] * (1.0 if w is None else w.reshape(-1)[a][:, None])
    return y


def gather_ref(y, pos, w):
    """(sum, sum of magnitudes) over the rows of each token."""
    T, k = pos.shape
    total, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for j in range(k):
        have = pos[:, j] >= 0
        v = y[pos[have, j]] * (1.0 if w is None else w[have, j][:, None])
        total[have] += v
        mag[have] += np.abs(v)
    return total, mag


def dots_ref(y, x, pos):
    T, k = pos.shape
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        have = pos[:, j] >= 0
        v = y[pos[have, j]] * x[have]
        dw[have, j], mag[have, j] = v.sum(1), np.abs(v).sum(1)
    return dw, mag


def rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


SHAPES = [  # T, H, k, S, absent
    (1, 1, 1, 1, 0.0), (1, 4096, 8, 230, 0.0), (3, 7, 2, 5, 0.0), (5, 8, 3, 3, 0.0),
    (64, 256, 4, 10, 0.0), (17, 1001, 4, 6, 0.3), (33, 513, 9, 40, 0.2), (9, 640, 17, 32, 0.1),
    (4, 96, 32, 64, 0.0), (130, 2048, 8, 3, 0.0), (2, 6144, 8, 16, 0.5), (7, 2051, 8, 16, 0.9),
    (300, 33, 5, 11, 0.1), (4100, 16, 8, 20, 0.05),
]


@pytest.mark.parametrize("T,k,S,absent", [(1, 1, 1, 0.0), (8, 8, 230, 0.0), (2048, 8, 166, 0.1),
                                          (2049, 8, 20, 0.3), (5000, 32, 64, 0.0)])
def test_positions(T, k, S, absent):
    from resident_expert_routing_amd import rows
    perm, _ = batch(T, k, S, seed=T + k, absent=absent)
    order = rows.RowOrder(torch.from_numpy(perm).cuda(), T, k)
    assert np.array_equal(order.pos.cpu().numpy(), reference(perm, T, k))
    assert np.array_equal(order.perm.cpu().numpy().reshape(-1), perm)


def test_positions_of_foreign_values():
    """Entries outside [0, n) name nothing; of an assignment named twice the later row stands."""
    from resident_expert_routing_amd import rows
    for n in (64, 40000):
        perm = np.full(n, -1, np.int32)
        perm[:6] = [3, n, 5, -7, 3, 2 ** 31 - 1]
        want = np.full(n, -1, np.int32)
        want[3], want[5] = 4, 2
        got = rows.RowOrder(torch.from_numpy(perm).cuda(), n // 4, 4).pos.cpu().numpy()
        assert np.array_equal(got.reshape(-1), want)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,H,k,S,absent", SHAPES)
@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_and_combine(T, H, k, S, absent, weighted, dtype):
    from resident_expert_routing_amd import rows
    perm, w = batch(T, k, S, seed=T * 31 + H, absent=absent)
    say(f"T={T} H={H} k={k} S={S} absent={absent} weighted={weighted} {dtype}")
    pos = reference(perm, T, k)
    order = rows.RowOrder(torch.from_numpy(perm).cuda(), T, k)
    wt = torch.from_numpy(w).cuda().requires_grad_() if weighted else None
    wn = w.astype(np.float64) if weighted else None
    live = perm >= 0

    # dispatch and its gradient
    x = rand((T, H), dtype, 1).requires_grad_()
    gy = rand((T * k, H), dtype, 2)
    y = rows.dispatch(x, order, wt)
    want = spread_ref(f64(x), perm, k, wn)
    assert np.all(f64(y)[~live] == 0)
    close(y, want, np.abs(want), 1 if weighted else 0, dtype, "dispatch")
    grads = torch.autograd.grad(y, [x] + ([wt] if weighted else []), gy)
    total, mag = gather_ref(f64(gy), pos, wn)
    close(grads[0], total, mag, k + 1, dtype, "dx")
    if weighted:
        dw, mag = dots_ref(f64(gy), f64(x), pos)
        close(grads[1], dw, mag, H + 12, None, "dispatch dw")
        assert np.all(f64(grads[1])[pos < 0] == 0)

    # combine and its gradient; rows that no assignment uses hold NaN and must not be seen
    r = rand((T * k, H), dtype, 3)
    r[torch.from_numpy(~live).cuda()] = float("nan")
    clean = np.where(live[:, None], f64(r), 0.0)
    r.requires_grad_()
    go = rand((T, H), dtype, 4)
    out = rows.combine(r, order, wt)
    total, mag = gather_ref(clean, pos, wn)
    close(out, total, mag, k + 1, dtype, "combine")
    grads = torch.autograd.grad(out, [r] + ([wt] if weighted else []), go)
    want = spread_ref(f64(go), perm, k, wn)
    assert np.all(f64(grads[0])[~live] == 0)
    close(grads[0], want, np.abs(want), 1 if weighted else 0, dtype, "drows")
    if weighted:
        dw, mag = dots_ref(clean, f64(go), pos)
        close(grads[1], dw, mag, H + 12, None, "combine dw")
        assert np.all(f64(grads[1])[pos < 0] == 0)


def test_gradients_against_differences():
    """Both calls are bilinear in (rows, weights), so a central difference of any
    step is exact up to rounding: d/ds <g, f(x + s v, w)> at s = 0."""
    from resident_expert_routing_amd import rows
    T, H, k, S = 23, 130, 4, 7
    perm, w = batch(T, k, S, seed=5, absent=0.2)
    order = rows.RowOrder(torch.from_numpy(perm).cuda(), T, k)
    wt = torch.from_numpy(w).cuda().requires_grad_()
    for f, n, m in ((rows.dispatch, T, T * k), (rows.combine, T * k, T)):
        x = rand((n, H), torch.float32, 1).requires_grad_()
        g = rand((m, H), torch.float32, 2)
        gx, gw = torch.autograd.grad(f(x, order, wt), [x, wt], g)
        v, u = rand((n, H), torch.float32, 3), rand((T, k), torch.float32, 4)
        with torch.no_grad():
            along = lambda a, b: float((f(a, order, b).double() * g.double()).sum())  # noqa: E731
            dx = (along(x + v, wt) - along(x - v, wt)) / 2
            dw = (along(x, wt + u) - along(x, wt - u)) / 2
        # 2^-24 rounding of ~H*n terms of size ~1, of random sign: 1e-4 is far above it
        scale = float(x.detach().double().norm() * g.double().norm())
        assert abs(dx - float((gx.double() * v.double()).sum())) <= 1e-5 * scale
        assert abs(dw - float((gw.double() * u.double()).sum())) <= 1e-5 * scale


def test_round_trip_is_exact():
    """Unweighted dispatch copies values: summing a power of two of copies is exact."""
    from resident_expert_routing_amd import rows
    T, H, k = 50, 77, 4
    perm, _ = batch(T, k, 9, seed=2)
    order = rows.RowOrder(torch.from_numpy(perm).cuda(), T, k)
    x = rand((T, H), torch.bfloat16, 1)
    x[3, 5], x[4, 6], x[5, 7] = float("inf"), float("nan"), 1e-40
    y = rows.combine(rows.dispatch(x, order), order)
    assert torch.equal(torch.nan_to_num(y, 7.0), torch.nan_to_num(4 * x, 7.0))


def test_infinities_and_nan_stay_in_their_rows():
    from resident_expert_routing_amd import rows
    T, H, k = 12, 200, 4
    perm, w = batch(T, k, 6, seed=3, absent=0.3)
    pos = reference(perm, T, k)
    order = rows.RowOrder(torch.from_numpy(perm).cuda(), T, k)
    wt = torch.from_numpy(w).cuda()
    r = rand((T * k, H), torch.float16, 1)
    clean = rows.combine(r, order, wt)
    t, j = np.argwhere(pos >= 0)[4]
    r[int(pos[t, j]), 9] = float("nan")
    r[int(pos[t, j]), 10] = float("-inf")
    out = rows.combine(r, order, wt)
    assert torch.isnan(out[t, 9]) and out[t, 10] == float("-inf")
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[t, 9:11] = False
    assert torch.equal(out[keep], clean[keep])
    # fp16 overflow of a sum is an infinity
    big = torch.full((T * k, H), 60000.0, dtype=torch.float16, device="cuda")
    s = f64(rows.combine(big, order))
    assert np.all(np.isinf(s[(pos >= 0).sum(1) > 1])) and np.all(s[(pos >= 0).sum(1) == 0] == 0)


def test_strides_and_layouts():
    """Rows inside a wider array at odd places, transposed and expanded tensors."""
    from resident_expert_routing_amd import rows
    T, H, k = 19, 75, 3
    perm, w = batch(T, k, 8, seed=6, absent=0.1)
    order = rows.RowOrder(torch.from_numpy(perm).cuda(), T, k)
    wt = torch.from_numpy(w).cuda()
    x = rand((T, H), torch.bfloat16, 1)
    want = rows.dispatch(x, order, wt)
    wide = torch.zeros(T, H + 9, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:3 + H] = x
    assert torch.equal(rows.dispatch(wide[:, 3:3 + H], order, wt), want)
    assert torch.equal(rows.dispatch(x.t().contiguous().t(), order, wt), want)
    one = x[:1].expand(T, H)
    assert torch.equal(rows.dispatch(one, order), rows.dispatch(one.contiguous(), order))
    # a broadcast gradient, as .sum() hands it back
    y = rand((T * k, H), torch.float32, 2).requires_grad_()
    rows.combine(y, order, wt).sum().backward()
    g = spread_ref(np.ones((T, H)), perm, k, w.astype(np.float64))
    assert np.array_equal(f64(y.grad), g)


def test_rows_behind_the_last_are_left_without_perm():
    """moe_dispatch without perm writes the rows that pos names and no others,
    and writes nothing between the rows of a wider output."""
    from resident_expert_routing_amd import binding as B
    T, H, k, pad = 11, 37, 4, 5
    perm, w = batch(T, k, 5, seed=8, absent=0.4)
    pos = torch.from_numpy(reference(perm, T, k).astype(np.int32)).cuda()
    x = rand((T, H), torch.float32, 1)
    out = torch.full((T * k, H + pad), 7.25, device="cuda")
    B.check(B.moe_dispatch(T, H, k, B.MOE_DT_FP32, pos, x, H, out, H + pad,
                           stream=torch.cuda.current_stream()))
    got = f64(out)
    live = perm >= 0
    assert np.all(got[:, H:] == 7.25) and np.all(got[~live] == 7.25)
    assert np.array_equal(got[live, :H], spread_ref(f64(x), perm, k, None)[live])


def test_empty_batch_and_absent_everything():
    from resident_expert_routing_amd import rows
    empty = rows.RowOrder(torch.empty(0, dtype=torch.int32, device="cuda"), 0, 4)
    x = torch.empty(0, 16, device="cuda", requires_grad=True)
    y = rows.combine(rows.dispatch(x, empty), empty)
    y.sum().backward()
    assert y.shape == (0, 16) and x.grad.shape == (0, 16)
    perm = torch.full((24,), -1, dtype=torch.int32, device="cuda")
    order = rows.RowOrder(perm, 6, 4)
    w = torch.ones(6, 4, device="cuda", requires_grad=True)
    x = rand((6, 16), torch.bfloat16, 1).requires_grad_()
    y = rows.dispatch(x, order, w)
    z = rows.combine(y, order, w)
    z.sum().backward()
    for t in (y, z, x.grad, w.grad):
        assert float(t.detach().abs().max()) == 0


def test_no_second_derivative():
    from resident_expert_routing_amd import rows
    order = rows.RowOrder(torch.arange(8, dtype=torch.int32, device="cuda"), 4, 2)
    x = rand((4, 16), torch.float32, 1).requires_grad_()
    w = torch.ones(4, 2, device="cuda", requires_grad=True)
    out = rows.combine(rows.dispatch(x, order), order, w)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(out.sum(), [x, w], create_graph=True)


def test_refusals():
    from resident_expert_routing_amd import rows
    perm = torch.zeros(8, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        rows.RowOrder(perm, 4, 3)
    with pytest.raises(ValueError):
        rows.RowOrder(perm.long(), 4, 2)
    with pytest.raises(ValueError):
        rows.RowOrder(perm, 4, 2, pos=perm.view(2, 4))
    order = rows.RowOrder(torch.arange(8, dtype=torch.int32, device="cuda"), 4, 2)
    for x, w in ((torch.zeros(5, 16, device="cuda"), None),
                 (torch.zeros(4, 16), None),
                 (torch.zeros(4, 16, device="cuda", dtype=torch.float64), None),
                 (torch.zeros(4, 16, device="cuda"), torch.zeros(4, 2)),
                 (torch.zeros(4, 16, device="cuda"), torch.zeros(3, 2, device="cuda")),
                 (torch.zeros(4, 16, device="cuda"), torch.zeros(2, 4, device="cuda")),
                 (torch.zeros(4, 16, device="cuda"),
                  torch.zeros(4, 2, device="cuda", dtype=torch.bfloat16)),
                 (torch.zeros(16, device="cuda"), None)):
        with pytest.raises(ValueError):
            rows.dispatch(x, order, w)
    with pytest.raises(ValueError):
        rows.combine(torch.zeros(4, 16, device="cuda"), order)


def test_another_stream_and_a_replayed_graph():
    """The calls follow the current stream, and a captured forward and backward
    gives the eager results on every replay, with new inputs and eager work between."""
    from resident_expert_routing_amd import rows
    T, H, k = 40, 264, 8
    perm, w = batch(T, k, 30, seed=9, absent=0.1)
    perm = torch.from_numpy(perm).cuda()

    def step(x, y, wt, g):
        order = rows.RowOrder(perm, T, k)
        r = rows.dispatch(x, order, wt)
        o = rows.combine(r + y, order, wt)
        return (r, o) + torch.autograd.grad(o, [x, y, wt], g)

    def inputs(seed):
        return [rand((T, H), torch.bfloat16, seed).requires_grad_(),
                rand((T * k, H), torch.bfloat16, seed + 1).requires_grad_(),
                (torch.from_numpy(w).cuda() * (1 + seed)).requires_grad_(),
                rand((T, H), torch.bfloat16, seed + 2)]

    want = [[t.detach().clone() for t in step(*inputs(s))] for s in range(4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(*inputs(0))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    del got

    held = inputs(0)
    with torch.cuda.stream(side):
        step(*held)
        side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step(*held)
    for s in (1, 2, 3, 0):
        with torch.no_grad():
            for h, v in zip(held, inputs(s)):
                h.copy_(v)
        torch.cuda.synchronize()
        graph.replay()
        eager = step(*inputs(s))
        torch.cuda.synchronize()
        for a, b, c in zip(out, want[s], eager):
            assert torch.equal(a, b) and torch.equal(b, c)


def test_backward_after_the_routing_buffers_are_reused():
    """The next batch's routing writes over perm (and over a pos of the caller's)
    before the backward pass of this one has run."""
    from resident_expert_routing_amd import rows
    T, H, k = 30, 100, 4
    perm, w = batch(T, k, 6, seed=12, absent=0.4)
    other, _ = batch(T, k, 6, seed=13)
    for own_pos in (False, True):
        buf = torch.from_numpy(perm).cuda()
        pos = torch.from_numpy(reference(perm, T, k).astype(np.int32)).cuda()
        order = rows.RowOrder(buf, T, k, pos=pos if own_pos else None)
        wt = torch.from_numpy(w).cuda().requires_grad_()
        x = rand((T, H), torch.float32, 1).requires_grad_()
        g = rand((T, H), torch.float32, 2)
        y = rows.dispatch(x, order, wt)
        out = rows.combine(y, order, wt)
        buf.copy_(torch.from_numpy(other))
        pos.copy_(torch.from_numpy(reference(other, T, k).astype(np.int32)))
        gy, gx = torch.autograd.grad(out, [y, x], g)
        want = spread_ref(f64(g), perm, k, w.astype(np.float64))
        close(gy, want, np.abs(want), 1, torch.float32, "drows")
        total, mag = gather_ref(want, reference(perm, T, k), w.astype(np.float64))
        close(gx, total, mag, k + 3, torch.float32, "dx")


@pytest.mark.parametrize("learned", [False, True])
def test_backward_after_the_weights_are_overwritten(learned):
    """The next batch's routing writes over sel_weight, unseen by torch, before the
    backward pass of this one has run."""
    from resident_expert_routing_amd import rows
    T, H, k = 30, 100, 4
    perm, w = batch(T, k, 6, seed=14, absent=0.4)
    order = rows.RowOrder(torch.from_numpy(perm).cuda(), T, k)
    wt = torch.from_numpy(w).cuda().requires_grad_(learned)
    x = rand((T, H), torch.float32, 1).requires_grad_()
    y = rand((T * k, H), torch.float32, 3).requires_grad_()
    g, gr = rand((T, H), torch.float32, 2), rand((T * k, H), torch.float32, 4)
    r, out = rows.dispatch(x, order, wt), rows.combine(y, order, wt)
    wt.data.fill_(7.0)
    gx = torch.autograd.grad(r, x, gr)[0]
    gy = torch.autograd.grad(out, y, g)[0]
    want = spread_ref(f64(g), perm, k, w.astype(np.float64))
    close(gy, want, np.abs(want), 1, torch.float32, "drows")
    total, mag = gather_ref(f64(gr), reference(perm, T, k), w.astype(np.float64))
    close(gx, total, mag, k + 3, torch.float32, "dx")


def test_two_calls_give_the_same_bits():
    from resident_expert_routing_amd import rows
    T, H, k = 257, 1024, 8
    perm, w = batch(T, k, 30, seed=10)
    order = rows.RowOrder(torch.from_numpy(perm).cuda(), T, k)
    r = rand((T * k, H), torch.bfloat16, 1).requires_grad_()
    wt = torch.from_numpy(w).cuda().requires_grad_()
    g = rand((T, H), torch.bfloat16, 2)
    first = torch.autograd.grad(rows.combine(r, order, wt), [r, wt], g)
    for _ in range(3):
        again = torch.autograd.grad(rows.combine(r, order, wt), [r, wt], g)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_offsets_past_32_bits():
    """Rows of more than 2^31 elements in all: the last ones are addressed right."""
    from resident_expert_routing_amd import rows
    T, H, k = 9000, 32768, 8                       # 2.36e9 elements of rows, 4.7 GB
    perm = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0).contiguous()
    order = rows.RowOrder(perm, T, k)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.arange(T, device="cuda").remainder(251).unsqueeze(1).expand(T, H))
    y = rows.dispatch(x, order)
    assert y.numel() > 2 ** 31
    p = torch.tensor([0, 1, T * k // 2, T * k - 2, T * k - 1], device="cuda")
    want = x[(perm[p] // k).long()]
    assert torch.equal(y[p], want)
    back = rows.combine(y, order)
    for t in (0, 1, T // 2, T - 1):
        assert torch.equal(back[t], 8 * x[t])
