"""moe_int8_quantize and moe_int8_matmul against their definitions in 64 bits on
the CPU, and the layer's experts in 8-bit integers against the same chain.

Quantised values and scales have to be equal: the definition fixes them (the
scale is a float32 division, whose float64 quotient rounded to float32 is the
same number, since 53 >= 2 * 24 + 2 bits make the second rounding harmless; the
integer is the rounded exact quotient, which float64 division finds, since two
24-bit numbers' quotient that is no half is at least 2^-50 of it away from one).

A product's integer sum is exact; it is rounded to float32 and scaled twice:
|y - exact| <= 3 * 2^-24 * |exact| (1 + 2^-22), then one rounding to the output
type.  With SwiGLU the gate value g carries that error d = 3 * 2^-24 |g|, which
silu, of slope at most 1.1, turns into 1.1 d |u|; exp(-g) is taken as 2^(-g
log2 e) with one rounding of the argument, |g| * 1.45 * 2^-24 of the result's
size, and 2 units in the last place of the instruction (4 * 2^-24); a sum (1), a
reciprocal to one unit (2) and two products (2) follow, and u's own error (3):
together at most (1.5 |g| + 12) * 2^-24 * |silu(g) u| more."""
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


def quantized(x):
    """(q, scale) by the definition, float64 numpy."""
    top = np.abs(x).max(axis=1)
    scale = np.maximum(top / 127.0, 2.0 ** -126).astype(np.float32)
    q = np.rint(x / scale.astype(np.float64)[:, None])
    return q.astype(np.int8), scale


def rows_of_all_sizes(M, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(2 * torch.randn(M, 1, generator=g))
    if M > 2:
        x[1] = 0
        x[2] = x[2].sign() * 3
    return x.to(dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M,K", [(1, 1), (8, 4096), (5, 15), (5, 16), (7, 17), (3, 1000), (64, 256),
                                 (300, 2048), (33, 2049), (9, 6144), (4, 8193), (2, 20001),
                                 (1030, 40)])
def test_quantize(M, K, dtype):
    from resident_expert_routing_amd import int8
    x = rows_of_all_sizes(M, K, dtype, M + K)
    q, scale = int8.quantize(x.cuda())
    wq, ws = quantized(x.double().numpy())
    assert np.array_equal(scale.cpu().numpy(), ws)
    assert np.array_equal(q.cpu().numpy(), wq)
    if K % 16:                                    # the padding of each row is zero
        whole = torch.as_strided(q, (M, (K + 15) // 16 * 16), (q.stride(0) if M > 1 else K, 1))
        assert int(whole[:, K:].abs().max()) == 0


def test_quantize_ties_and_halves():
    """Scale exactly 1, 2 and 3/127: quotients on and next to a half, both signs."""
    from resident_expert_routing_amd import int8
    halves = np.arange(-126.5, 127, 1.0)
    near = np.concatenate([np.nextafter(np.float32(halves), np.float32(s)) for s in (-500, 500)])
    base = np.concatenate([halves, near, [127.0, -127.0, 0.0, -0.0]]).astype(np.float32)
    x = np.stack([base, 2 * base, base * np.float32(3 / 127), base * np.float32(2.0 ** -100)])
    q, s = int8.quantize(torch.from_numpy(x).cuda())
    wq, ws = quantized(x.astype(np.float64))
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), wq)


def test_quantize_extremes():
    from resident_expert_routing_amd import int8
    big, tiny = torch.finfo(torch.float32).max, 2.0 ** -149
    x = torch.zeros(7, 50)
    x[0, 3], x[0, 4] = big, -big / 3              # the largest values
    x[1, 7] = tiny                                # a subnormal row: scale 2^-126, values 0
    x[2, 1], x[2, 2] = 2.0 ** -126 * 127, 2.0 ** -126 * 1.5
    x[3, 9] = float("inf")
    x[4, 9] = float("nan")
    x[5, 9], x[5, 8] = float("-inf"), float("nan")
    q, s = int8.quantize(x.cuda())
    q, s = q.cpu(), s.cpu()
    fine = [0, 1, 2, 6]
    wq, ws = quantized(x[fine].double().numpy())
    assert np.array_equal(s[fine].numpy(), ws) and np.array_equal(q[fine].numpy(), wq)
    assert torch.isnan(s[3:6]).all() and int(q[3:6].abs().max()) == 0
    assert int(q[0, 3]) == 127 and int(q[2, 2]) == 2


def test_quantize_strides_and_given_outputs():
    from resident_expert_routing_amd import int8
    x = rows_of_all_sizes(21, 100, torch.bfloat16, 3).cuda()
    q, s = int8.quantize(x)
    wide = torch.zeros(21, 131, dtype=torch.bfloat16, device="cuda")
    wide[:, 5:105] = x
    q2, s2 = int8.quantize(wide[:, 5:105])
    assert torch.equal(q, q2) and torch.equal(s, s2)
    q3, s3 = int8.quantize(x.t().contiguous().t())
    assert torch.equal(q, q3) and torch.equal(s, s3)
    room = torch.full((21, 160), 77, dtype=torch.int8, device="cuda")
    out = (room[:, 16:116], torch.empty(21, device="cuda"))
    got = int8.quantize(x, out)
    assert got[0] is out[0] and torch.equal(got[0], q) and torch.equal(got[1], s)
    assert bool((room[:, :16] == 77).all()) and bool((room[:, 128:] == 77).all())
    assert int8.quantize(x[:0])[0].shape == (0, 100)
    with pytest.raises(ValueError):
        int8.quantize(x, (room[:, 8:108], out[1]))
    with pytest.raises(ValueError):
        int8.quantize(x.double())
    with pytest.raises(ValueError, match="gradient"):
        int8.quantize(x.clone().requires_grad_())


def ints(shape, seed, low=-127):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(low, 128, shape, generator=g, dtype=torch.int8)


def scales(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.rand(shape, generator=g) * 2e-3 + 1e-4


def reference(a, sa, b, sb, offsets, index, div, swiglu, out):
    """(values, error bounds before the last rounding); `out` gives the rows left alone."""
    a, sa, sb = a.double().numpy(), sa.double().numpy(), sb.double().numpy()
    M, N = out.shape
    want, err = out.double().numpy().copy(), np.zeros((M, N))
    seen = np.zeros(M, bool)
    edges = [0, M] if offsets is None else offsets
    for g in range(len(edges) - 1):
        for_g = np.arange(edges[g], edges[g + 1])
        r = for_g if index is None else np.where(index[for_g] < 0, -1, index[for_g] // div)
        ok = (r >= 0) & (r < a.shape[0])
        for_g, r = for_g[ok], r[ok]
        if not len(r):
            continue
        bg, sg = (b, sb) if offsets is None else (b[g], sb[g])
        z = (a[r] @ bg.double().numpy().T) * sa[r][:, None] * sg
        if swiglu:
            gate, up = z[:, :N], z[:, N:]
            si = gate / (1 + np.exp(-gate))
            want[for_g] = si * up
            err[for_g] = 1.1 * 3 * 2.0 ** -24 * np.abs(gate * up) + \
                (1.5 * np.abs(gate) + 12) * 2.0 ** -24 * np.abs(si * up)
        else:
            want[for_g] = z
            err[for_g] = 3.01 * 2.0 ** -24 * np.abs(z)
        seen[for_g] = True
    return want, err, seen


def check(M, N, K, *, G=0, swiglu=False, index=None, index_div=1, a_rows=None, offsets=None,
          dtype=torch.bfloat16, seed=0, low=-127):
    from resident_expert_routing_amd import int8
    wide = 2 * N if swiglu else N
    a_rows = M if a_rows is None else a_rows
    a, b = ints((a_rows, K), seed, low), ints((G, wide, K) if G else (wide, K), seed + 1, low)
    sa, sb = scales((a_rows,), seed + 2), scales((G, wide) if G else (wide,), seed + 3)
    out = torch.full((M, N), -3.5, dtype=dtype)
    dev = lambda t: None if t is None else torch.as_tensor(t).cuda()  # noqa: E731
    got = int8.matmul(int8.pad_rows(a.cuda()), sa.cuda(), int8.pad_rows(b.cuda()), sb.cuda(),
                      offsets=dev(None if offsets is None else np.asarray(offsets, np.int32)),
                      index=dev(None if index is None else np.asarray(index, np.int32)),
                      index_div=index_div, swiglu=swiglu, out=out.cuda())
    want, err, seen = reference(a, sa, b, sb, offsets, index, index_div, swiglu, out)
    got = got.cpu().double().numpy()
    bound = err * 1.01 + torch.finfo(dtype).eps / 2 * (np.abs(want) + err) + UNDER[dtype]
    assert np.array_equal(got[~seen], want[~seen]), "rows of no group were written"
    off = np.abs(got - want)
    assert np.all(off[seen] <= bound[seen]), float(np.max(off[seen] / bound[seen]))
    return got


SIZES = [(1, 1, 1), (1, 16, 15), (2, 33, 16), (5, 31, 17), (16, 32, 63), (17, 48, 64), (3, 100, 65),
         (64, 64, 256), (65, 130, 200), (1, 4096, 4096), (8, 500, 1000), (130, 257, 129),
         (257, 300, 384), (300, 512, 1111), (513, 640, 640), (1, 257, 6144), (100, 1000, 2064)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_dense(M, N, K, swiglu, dtype):
    say(f"dense M={M} N={N} K={K} swiglu={swiglu} {dtype}")
    check(M, N, K, swiglu=swiglu, dtype=dtype, seed=M + N + K)


GROUPS = [  # sizes of the groups
    [1], [0, 3, 0, 0, 1, 0], [5] * 70, [0] * 40 + [64] + [0] * 200, [17, 0, 16, 15, 33, 1, 0, 129],
    [300, 2, 0, 70], [1] * 8, [0, 0, 0], [257, 256, 255], [600, 1, 0, 0, 513],
]


@pytest.mark.parametrize("sizes", GROUPS, ids=lambda s: f"{len(s)}x{sum(s)}")
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("behind", [0, 9])
def test_grouped(sizes, swiglu, behind):
    """Groups of every size, empty ones among them, and rows behind the last group."""
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    M = int(offsets[-1]) + behind
    if M == 0:
        pytest.skip("no rows at all")
    say(f"groups of {sizes[:8]}... M={M} swiglu={swiglu}")
    for N, K in ((48, 96), (130, 320), (33, 77)):
        check(M, N, K, G=len(sizes), offsets=offsets, swiglu=swiglu, seed=M + N)


# Products of many tiles take another kernel form than those of few: here every
# height of a tile (64, 128, 192, 256, 320 rows) and both sides of each, and K
# of one stage (128) and several, cut and whole.
HEIGHTS = [1, 63, 64, 65, 0, 128, 129, 192, 193, 256, 257, 320, 321, 400, 3]


@pytest.mark.parametrize("K", [1, 16, 77, 128, 130, 257, 384, 515])
@pytest.mark.parametrize("swiglu", [False, True])
def test_tiled_groups(K, swiglu):
    offsets = np.concatenate([[0], np.cumsum(HEIGHTS)])
    M = int(offsets[-1]) + 5
    N = 1801 if swiglu else 3301
    say(f"tiles K={K} swiglu={swiglu}")
    dtype = DTYPES[K % 3]
    check(M, N, K, G=len(HEIGHTS), offsets=offsets, swiglu=swiglu, dtype=dtype, seed=K)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_tiled_rows_by_index(swiglu, dtype):
    """As test_rows_by_index, in tiles; more groups than a wave keeps in registers."""
    rng = np.random.default_rng(4)
    for G in (40, 300):
        sizes = rng.integers(0, 12 if G > 100 else 90, G)
        offsets = np.concatenate([[0], np.cumsum(sizes)])
        M, k = int(offsets[-1]) + 8, 4
        index = rng.permutation(M).astype(np.int32)
        index[[3, 40, M - 1]] = [-1, M * k + 5, -2 ** 31]
        check(M, 640, 300, G=G, offsets=offsets, index=index, index_div=k, a_rows=(M + k - 1) // k,
              swiglu=swiglu, dtype=dtype, seed=G)


@pytest.mark.parametrize("G,M", [(257, 40), (300, 41), (8192, 40), (8192, 9000), (256, 700)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_many_groups(G, M, swiglu):
    """More groups than a wave keeps in registers (256), to the most there can be;
    most of them empty, the first and the last in use."""
    rng = np.random.default_rng(G + M)
    sizes = np.zeros(G, int)
    sizes[0], sizes[-1] = 3, 2
    for g in rng.integers(0, G, M - 5):
        sizes[g] += 1
    check(M, 64, 80, G=G, offsets=np.concatenate([[0], np.cumsum(sizes)]), swiglu=swiglu, seed=G)


@pytest.mark.parametrize("M,N,K", [(160, 4200, 200), (257, 3333, 129), (513, 2570, 64),
                                   (1030, 900, 333), (3200, 300, 96), (2081, 1030, 1000)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_tiled_dense(M, N, K, swiglu):
    say(f"dense tiles M={M} N={N} K={K} swiglu={swiglu}")
    check(M, N, K, swiglu=swiglu, dtype=DTYPES[M % 3], seed=M)


def test_tiled_layouts_and_foreign_offsets():
    """Strides, what lies behind rows, and offsets that are no bucketing, in tiles."""
    from resident_expert_routing_amd import int8
    N, K, sizes = 2600, 200, [300, 0, 390, 20, 5, 70, 129, 64, 0, 1, 200, 33, 40, 8, 8, 8, 8, 8]
    G, M = len(sizes), sum(sizes)
    offsets = torch.as_tensor(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
    a, b = ints((M, K), 1).cuda(), int8.pad_rows(ints((G, N, K), 2).cuda())
    sa, sb = scales((M,), 3).cuda(), scales((G, N), 4).cuda()
    want = int8.matmul(a, sa, b, sb, offsets=offsets)
    big_b = torch.full((G, N + 3, 288), 99, dtype=torch.int8, device="cuda")
    big_b[:, 1:1 + N, 32:32 + K] = b
    big_a = torch.full((M, 272), -99, dtype=torch.int8, device="cuda")
    big_a[:, 16:16 + K] = a
    room = torch.full((M + 64, N + 5), 9.0, dtype=torch.bfloat16, device="cuda")
    got = int8.matmul(big_a[:, 16:16 + K], sa, big_b[:, 1:1 + N, 32:32 + K], sb, offsets=offsets,
                      out=room[32:32 + M, 3:3 + N])
    assert torch.equal(got, want)
    edge = room.clone()
    edge[32:32 + M, 3:3 + N] = 9
    assert bool((edge == 9).all())
    wild = offsets.clone()
    wild[0], wild[-1], wild[-2] = -3, 2 ** 31 - 1, M + 70
    room.fill_(9)
    int8.matmul(a, sa, b, sb, offsets=wild, out=room[32:32 + M, 3:3 + N])
    room[32:32 + M, 3:3 + N] = 9
    assert bool((room == 9).all())


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("sizes", [[7, 0, 20, 1, 36], [200, 100, 0, 300, 40]])
def test_rows_by_index(sizes, swiglu):
    """Rows named by assignment, some naming nothing or something outside a."""
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    M = int(offsets[-1]) + 8
    k = 4
    rng = np.random.default_rng(3)
    index = rng.permutation(M).astype(np.int32)
    index[[3, 40, M - 1]] = [-1, M * k + 5, -2 ** 31]
    index[17] = index[18]                          # the same row twice
    check(M, 72, 208, G=len(sizes), offsets=offsets, index=index, index_div=k,
          a_rows=(M + k - 1) // k, swiglu=swiglu, seed=5)


@pytest.mark.parametrize("sizes", [[7, 0, 20, 1, 36], [200, 100, 0, 300, 40]])
def test_offsets_that_are_no_bucketing(sizes):
    """Offsets past M are cut; nothing outside out is written (rows around it keep their value)."""
    from resident_expert_routing_amd import int8
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    M = int(offsets[-1]) - 5
    offsets[0] = -3
    room = torch.full((M + 64, 48), 2.5, device="cuda")
    a, b = ints((M, 64), 1).cuda(), ints((5, 48, 64), 2).cuda()
    int8.matmul(a, scales((M,), 3).cuda(), b, scales((5, 48), 4).cuda(),
                offsets=torch.as_tensor(offsets.astype(np.int32)).cuda(), out=room[32:32 + M])
    room = room.cpu()
    assert bool((room[:32] == 2.5).all()) and bool((room[32 + M:] == 2.5).all())
    assert not bool((room[32:32 + M] == 2.5).any())


def test_whole_range_of_the_integers():
    """-128 and sums past 2^24, where the integer sum is no float32."""
    check(40, 64, 4096, low=-128, seed=1, dtype=torch.float32)
    from resident_expert_routing_amd import int8
    K = 131056
    a = torch.full((20, K), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(20, device="cuda")
    for M in (1, 20):
        y = int8.matmul(a[:M], one[:M], a, one, out_dtype=torch.float32)
        assert bool((y == float(128 * 128 * K)).all())
    a, one = a[:1].repeat(3100, 1), torch.ones(3100, device="cuda")       # in tiles
    y = int8.matmul(a, one, a[:32], one[:32], out_dtype=torch.float32)
    assert bool((y == float(128 * 128 * K)).all())


def test_layouts():
    """Matrices with strides of their own, groups apart as in an arena, out inside a wider array."""
    from resident_expert_routing_amd import int8
    for M, sizes in ((50, [20, 0, 25]), (700, [300, 390, 0])):
        N, K, G = 72, 100, 3
        offsets = torch.as_tensor(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
        a, b = ints((M, K), 1).cuda(), ints((G, N, K), 2).cuda()
        sa, sb = scales((M,), 3).cuda(), scales((G, N), 4).cuda()
        want = int8.matmul(a, sa, int8.pad_rows(b), sb, offsets=offsets,
                           out=torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"))
        big_b = torch.full((G, N + 3, 160), 99, dtype=torch.int8, device="cuda")
        big_b[:, 1:1 + N, 32:32 + K] = b
        big_a = torch.full((M, 144), -99, dtype=torch.int8, device="cuda")
        big_a[:, 16:16 + K] = a                    # what follows a row's K elements is no zero
        big_s = torch.zeros(G, N + 7, device="cuda")
        big_s[:, 2:2 + N] = sb
        room = torch.full((M, N + 5), 9.0, dtype=torch.bfloat16, device="cuda")
        room[:, 3:3 + N] = 0
        got = int8.matmul(big_a[:, 16:16 + K], sa, big_b[:, 1:1 + N, 32:32 + K],
                          big_s[:, 2:2 + N], offsets=offsets, out=room[:, 3:3 + N])
        assert torch.equal(got, want)
        assert bool((room[:, :3] == 9).all()) and bool((room[:, 3 + N:] == 9).all())
    with pytest.raises(ValueError):
        int8.matmul(a, sa, b, sb, offsets=offsets)             # b is not laid out
    with pytest.raises(ValueError):
        int8.matmul(a, sa, int8.pad_rows(b), sb)               # groups without offsets
    with pytest.raises(ValueError):
        int8.matmul(a, sa[1:], int8.pad_rows(b[0]), sb[0])
    with pytest.raises(ValueError):
        int8.matmul(a, sa, int8.pad_rows(b[0]), sb[0], out_dtype=torch.float64)
    with pytest.raises(ValueError):
        int8.matmul(a, sa, int8.pad_rows(b[0][:71]), sb[0][:71], swiglu=True)
    with pytest.raises(ValueError):
        int8.matmul(a, sa.double(), int8.pad_rows(b[0]), sb[0])
    with pytest.raises(ValueError):
        int8.matmul(a, sa, int8.pad_rows(b), sb, offsets=offsets.long())
    with pytest.raises(ValueError):
        int8.matmul(a, sa, int8.pad_rows(b), sb, offsets=offsets, index=offsets.cpu())
    with pytest.raises(ValueError):
        int8.matmul(a, sa, int8.pad_rows(b), sb, offsets=offsets, out=a.float())


def test_scales_that_are_nan_reach_only_their_row():
    from resident_expert_routing_amd import int8
    x = rows_of_all_sizes(9, 96, torch.float32, 1)
    x[4, 2] = float("nan")
    q, s = int8.quantize(x.cuda())
    b = ints((40, 96), 2).cuda()
    y = int8.matmul(q, s, b, scales((40,), 3).cuda(), out_dtype=torch.float32).cpu()
    assert torch.isnan(y[4]).all() and torch.isfinite(y[[0, 1, 2, 3, 5, 6, 7, 8]]).all()


def test_streams_and_replayed_graph():
    from resident_expert_routing_amd import int8
    for M, N in ((6, 80), (900, 80), (900, 6200)):
        K, G = 272, 4
        sizes = [M // 3, 0, M // 2, M - M // 3 - M // 2]
        off = torch.as_tensor(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
        b, sb = ints((G, 2 * N, K), 2).cuda(), scales((G, 2 * N), 4).cuda()
        x = rows_of_all_sizes(M, K, torch.bfloat16, 7).cuda()

        def step():
            q, s = int8.quantize(x)
            return q, s, int8.matmul(q, s, b, sb, offsets=off, swiglu=True)

        want = step()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = step()
        side.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = step()
        for seed in (8, 9, 10):
            x.copy_(rows_of_all_sizes(M, K, torch.bfloat16, seed))
            torch.cuda.synchronize()
            graph.replay()
            eager = step()
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(held, eager))


def test_offsets_past_32_bits():
    """A group's matrix and rows of out more than 2^31 bytes into their arrays."""
    from resident_expert_routing_amd import int8
    G, N, K = 40, 8192, 8192                        # 2.7 GB of weights
    b = torch.zeros(G, N, K, dtype=torch.int8, device="cuda")
    b[G - 1] = ints((N, K), 1).cuda()
    sb = torch.ones(G, N, device="cuda")
    for m in (3, 300):
        a = ints((m, K), 2).cuda()
        off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
        off[G] = m
        y = int8.matmul(a, torch.ones(m, device="cuda"), b, sb, offsets=off,
                        out_dtype=torch.float32)
        want = a.cpu().double() @ b[G - 1, ::1021].cpu().double().t()
        assert float((y[:, ::1021].cpu().double() - want).abs().max()) <= \
            3 * 2.0 ** -24 * float(want.abs().max())


def routed(T, H, E, k, I, S, resident, seed):
    """moe_route's bucketing of a random batch, and floating experts for its slots."""
    from resident_expert_routing_amd import runtime as R
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, H, generator=g)).to(torch.bfloat16).cuda()
    w_router = (torch.randn(E, H, generator=g) / H ** 0.5).cuda()
    slot = torch.full((E,), -1, dtype=torch.int32)
    slot[torch.randperm(E, generator=g)[:resident]] = torch.randperm(S, generator=g)[:resident].int()
    buf = R.LayerBuffers(T, H, E, k, I, S, torch.device("cuda", 0))
    R.route(buf, x.view(torch.int16), w_router, None, slot.cuda(), torch.cuda.current_stream())
    weights = [(torch.randn(S, *shape, generator=g) * shape[1] ** -0.5).cuda()
               for shape in ((I, H), (I, H), (H, I))]
    return buf, x, weights, (w_router, slot.cuda())


@pytest.mark.parametrize("T,H,E,k,I,S,resident", [
    (1, 256, 16, 4, 128, 10, 10), (8, 512, 64, 8, 256, 40, 40), (9, 256, 16, 4, 96, 10, 3),
    (64, 256, 16, 4, 128, 10, 10), (600, 512, 32, 8, 384, 24, 24), (300, 320, 8, 2, 160, 8, 5)])
def test_layer_in_int8(T, H, E, k, I, S, resident):
    """Routing, int8 experts and combine together: against the same chain in
    float64 with the quantised weights and activations.  Where the two chains'
    bf16 values of h differ by a rounding, a quantised value of h can differ by
    one step; the layer's bar (relative L2 of 5e-3, which holds MXFP4's own
    differences of that kind) covers it and the last rounding."""
    from resident_expert_routing_amd import int8, rows
    from resident_expert_routing_amd import runtime as R
    buf, x, (wg, wu, wd), route_args = routed(T, H, E, k, I, S, resident, T + H)
    ex = int8.Int8Experts.from_weights(wg, wu, wd)
    out = ex.forward(x, buf.slot_offsets, buf.perm, buf.sel_weight)
    say(f"T={T} H={H} I={I} S={S}: {int(buf.slot_offsets[-1])} of {T * k} picks have a slot")

    deq = lambda q, s: q.cpu().double().numpy() * s.cpu().double().numpy()[..., None]  # noqa: E731
    gu, dn = deq(ex.gate_up, ex.gate_up_scale), deq(ex.down, ex.down_scale)
    a, sa = quantized(x.cpu().double().numpy())
    a = a * sa.astype(np.float64)[:, None]
    off, perm = buf.slot_offsets.cpu().numpy(), buf.perm.cpu().numpy()
    w = buf.sel_weight.cpu().double().numpy().reshape(-1)
    want = np.zeros((T, H))
    for s in range(S):
        for p in range(off[s], off[s + 1]):
            z = gu[s] @ a[perm[p] // k]
            h = torch.from_numpy(z[:I] / (1 + np.exp(-z[:I])) * z[I:]).to(torch.bfloat16)
            hq, hs = quantized(h.double().numpy()[None])
            y = torch.from_numpy(dn[s] @ (hq[0] * float(hs[0]))).to(torch.bfloat16).double().numpy()
            want[perm[p] // k] += w[perm[p]] * y
    got = out.cpu().double().numpy()
    if not want.any():
        assert not got.any()
        return
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    say(f"  relative L2 {rel:.2e}")
    assert rel <= 5e-3
    none = (buf.sel_slot.cpu().numpy() < 0).all(axis=1)
    assert np.all(got[none] == 0)
    # the whole step of the runtime, and the same layer with the rows brought into
    # order first, as other experts would take them
    hist = torch.zeros(E, dtype=torch.float64, device="cuda")
    step = R.layer_step_int8(buf, x, route_args[0], None, route_args[1], hist, ex)
    assert torch.equal(step, out) and float(hist.sum()) > 0
    order = rows.RowOrder(buf.perm, T, k)
    q, s = int8.quantize(rows.dispatch(x, order))
    h = int8.matmul(q, s, ex.gate_up, ex.gate_up_scale, offsets=buf.slot_offsets, swiglu=True)
    y = int8.matmul(*int8.quantize(h), ex.down, ex.down_scale, offsets=buf.slot_offsets)
    assert torch.equal(rows.combine(y, order, buf.sel_weight), out)


def test_experts_of_an_empty_batch():
    from resident_expert_routing_amd import int8
    ex = int8.Int8Experts.empty(3, 64, 32, torch.device("cuda", 0))
    out = ex.forward(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                     torch.zeros(4, dtype=torch.int32, device="cuda"),
                     torch.empty(0, dtype=torch.int32, device="cuda"),
                     torch.empty(0, 2, device="cuda"))
    assert out.shape == (0, 64)


def test_training_through_the_routing():
    """dispatch, floating experts in torch and combine: gradients of the rows, the
    experts and the routing weights against float64 autograd on the CPU."""
    from resident_expert_routing_amd import rows
    T, H, E, k, I, S = 48, 128, 16, 4, 64, 12
    buf, x, (wg, wu, wd), _ = routed(T, H, E, k, I, S, 12, 1)
    off = buf.slot_offsets.tolist()

    def layer(x, w, wg, wu, wd, dispatch, combine):
        r = dispatch(x)
        ys = []
        for s in range(S):
            v = r[off[s]:off[s + 1]]
            ys.append((torch.nn.functional.silu(v @ wg[s].t()) * (v @ wu[s].t())) @ wd[s].t())
        ys.append(r[off[S]:])
        return combine(torch.cat(ys), w)

    order = rows.RowOrder(buf.perm, T, k)
    ins = [x.float(), buf.sel_weight, wg, wu, wd]
    mine = [t.detach().clone().requires_grad_() for t in ins]
    g = torch.randn(T, H, generator=torch.Generator().manual_seed(2))
    out = layer(*mine, lambda x: rows.dispatch(x, order), lambda r, w: rows.combine(r, order, w))
    got = torch.autograd.grad(out, mine, g.cuda())

    theirs = [t.detach().cpu().double().requires_grad_() for t in ins]
    perm, pos = buf.perm.cpu().long(), order.pos.cpu().long()
    ref = layer(*theirs, lambda x: x[perm // k],
                lambda r, w: (r[pos] * w.unsqueeze(2)).sum(1))
    want = torch.autograd.grad(ref, theirs, g.double())
    # float32 matrix products over at most 128 terms: errors of 128 * 2^-24 per product, three deep
    ref = ref.detach()
    assert float((out.detach().cpu().double() - ref).abs().max()) <= 1e-4 * float(ref.abs().max())
    for u, v in zip(got, want):
        assert float((u.cpu().double() - v).norm()) <= 1e-4 * float(v.norm())


def test_outputs_given_and_gradients():
    """A given output counts as changed, so that a backward pass that needs what it
    held before is refused; outputs and scales that want a gradient are refused."""
    from resident_expert_routing_amd import int8, rows
    q, s = int8.quantize(torch.randn(8, 64, device="cuda"))
    wq, ws = int8.quantize(torch.randn(32, 64, device="cuda"))
    out = torch.empty(8, 32, device="cuda")
    order = rows.RowOrder(torch.arange(8, dtype=torch.int32, device="cuda"), 4, 2)
    w = torch.ones(4, 2, device="cuda", requires_grad=True)
    y = rows.combine(int8.matmul(q, s, wq, ws, out=out), order, w)
    int8.matmul(q, s, wq, ws, out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    before = q._version, s._version
    int8.quantize(torch.randn(8, 64, device="cuda"), (q, s))
    assert q._version > before[0] and s._version > before[1]
    with torch.inference_mode():
        held = torch.empty(8, 32, device="cuda")
        int8.matmul(q, s, wq, ws, out=held)

    def wanting(t):
        return t.detach().clone().requires_grad_()

    for args, kw in (((q, wanting(s), wq, ws), {}), ((q, s, wq, wanting(ws)), {}),
                     ((q, s, wq, ws), dict(out=wanting(out)))):
        with pytest.raises(ValueError, match="gradient"):
            int8.matmul(*args, **kw)
        with torch.no_grad():
            int8.matmul(*args, **kw)
    with pytest.raises(ValueError, match="gradient"):
        int8.quantize(torch.randn(8, 64, device="cuda"), (q, wanting(s)))
