"""Row operators at the edges of what their header allows: the largest batches,
assignments named twice, tensors that carry a tangent."""
import pytest
import torch

from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import resident_expert_routing_amd  # noqa: F401
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_the_most_assignments_there_can_be():
    """T*k = 2^31 - 1 tokens of one element: each is moved once, to the reversed
    row and back, with its dot product (values are exact in bf16)."""
    from resident_expert_routing_amd import binding as B
    n = 2 ** 31 - 1
    say(f"rows of {n} tokens")
    pos = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")
    x = torch.arange(n, dtype=torch.int32, device="cuda").remainder_(251).to(torch.bfloat16)
    y, z = torch.full_like(x, -1.0), torch.full_like(x, -1.0)
    stream = torch.cuda.current_stream()
    dt = B.MOE_DT_BF16
    B.check(B.moe_dispatch(n, 1, 1, dt, pos, x, 1, y, 1, stream=stream))
    assert torch.equal(y.flip(0), x)
    B.check(B.moe_combine(n, 1, 1, dt, pos, y, 1, z, 1, stream=stream))
    assert torch.equal(z, x)
    two = torch.full_like(x, 2.0)
    dw = torch.full((n,), -1.0, device="cuda")
    z.fill_(-1.0)
    B.check(B.moe_dispatch_backward(n, 1, 1, dt, pos, y, 1, z, 1, other=two, other_stride=1,
                                    dweight=dw, stream=stream))
    assert torch.equal(z, x) and torch.equal(dw.to(torch.bfloat16), 2 * x)
    z.fill_(-1.0)
    dw.fill_(-1.0)
    B.check(B.moe_combine_backward(n, 1, 1, dt, pos, two, 1, z, 1, other=y, other_stride=1,
                                   dweight=dw, stream=stream))
    assert torch.equal(z, two) and torch.equal(dw.to(torch.bfloat16), 2 * x)


@pytest.mark.parametrize("T,H,k", [(4, 3, 2), (9, 96, 8), (33, 1001, 9), (2000, 40, 4)])
@pytest.mark.parametrize("grad", [False, True])
def test_an_assignment_named_twice(T, H, k, grad):
    """Its row is the later one; the earlier one belongs to nobody and is zero,
    in dispatch and in combine's backward pass, whatever the output held before."""
    from resident_expert_routing_amd import binding as B
    n = T * k
    g = torch.Generator().manual_seed(T)
    perm = torch.randperm(n, generator=g).to(torch.int32)
    perm[n // 2] = perm[n - 1]                # one twice, so another one not at all
    perm[1] = perm[n - 2]
    perm[0] = -1
    pos = torch.full((n,), -1, dtype=torch.int32)
    for p in range(n):
        if perm[p] >= 0:
            pos[perm[p]] = p
    owned = torch.zeros(n, dtype=torch.bool)
    owned[pos[pos >= 0].long()] = True
    x, w = torch.randn(T, H, generator=g), torch.rand(T, k, generator=g)
    other = torch.randn(n, H, generator=g)
    out = torch.full((n, H), 7.25, device="cuda")
    dw = torch.full((T, k), -1.0, device="cuda")
    dperm, dpos = perm.cuda(), torch.empty(T, k, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream()
    B.check(B.moe_positions(dperm, T, k, dpos, stream=stream))
    assert torch.equal(dpos.cpu().view(-1), pos)
    args = (T, H, k, B.MOE_DT_FP32, dpos, x.cuda(), H, out, H, w.cuda())
    if grad:
        B.check(B.moe_combine_backward(*args, perm=dperm, other=other.cuda(), other_stride=H,
                                       dweight=dw, stream=stream))
        dots = torch.where(pos < 0, 0.0, (other[pos.clamp(min=0).long()].double()
                                          * x.double().repeat_interleave(k, 0)).sum(1))
        mag = (other[pos.clamp(min=0).long()].double()
               * x.double().repeat_interleave(k, 0)).abs().sum(1)
        off = (dw.cpu().view(-1).double() - dots).abs()
        assert bool((off <= (H + 12) * 2.0 ** -24 * mag).all())
    else:
        B.check(B.moe_dispatch(*args, perm=dperm, stream=stream))
    a = perm.clamp(min=0).long()
    # one float32 product: the same number on both sides
    want = torch.where(owned[:, None], x[a // k] * w.view(-1)[a][:, None], 0.0)
    assert torch.equal(out.cpu(), want)


def test_tangents_are_refused():
    """No call drops a forward-mode derivative: of the rows, of the weights, with
    and without gradients recorded, nor of the gradient in a backward pass."""
    from torch.autograd import forward_ad
    from resident_expert_routing_amd import int8, rows
    T, H, k = 6, 32, 2
    order = rows.RowOrder(torch.randperm(T * k, device="cuda").int(), T, k)
    ins = {"x": torch.randn(T, H, device="cuda"), "r": torch.randn(T * k, H, device="cuda"),
           "w": torch.rand(T, k, device="cuda")}
    q, s = int8.quantize(ins["x"])
    wq, ws = int8.quantize(torch.randn(8, H, device="cuda"))
    out = torch.empty(T, 8, device="cuda")
    calls = [
        (lambda x: rows.dispatch(x, order), ins["x"]),
        (lambda x: rows.dispatch(x, order, ins["w"]), ins["x"]),
        (lambda w: rows.dispatch(ins["x"], order, w), ins["w"]),
        (lambda r: rows.combine(r, order, ins["w"]), ins["r"]),
        (lambda w: rows.combine(ins["r"], order, w), ins["w"]),
        (int8.quantize, ins["x"]),
        (lambda t: int8.quantize(ins["x"], (q, t)), s),
        (lambda t: int8.matmul(q, t, wq, ws), s),
        (lambda t: int8.matmul(q, s, wq, t), ws),
        (lambda t: int8.matmul(q, s, wq, ws, out=t), out),
    ]
    for call, t in calls:
        for wants in (False, True):
            with forward_ad.dual_level():
                u = t.detach().clone().requires_grad_(wants)
                d = forward_ad.make_dual(u, torch.ones_like(u))
                with pytest.raises(ValueError, match="tangent|gradient"):
                    call(d)
                with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
                    call(d)
            with torch.no_grad():
                call(t.detach().clone())
    x = ins["x"].detach().clone().requires_grad_()
    w = ins["w"].detach().clone().requires_grad_()
    y = rows.dispatch(x, order, w)
    g = torch.ones_like(y)
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="tangent"):
            torch.autograd.grad(y, [x, w], forward_ad.make_dual(g, g), retain_graph=True)
        torch.autograd.grad(y, [x, w], g)


def test_sizes_past_32_bits_are_refused():
    """Sizes that a C int would cut: refused before anything is copied or written."""
    from resident_expert_routing_amd import int8, rows
    from resident_expert_routing_amd.binding import MoeError
    wide = 2 ** 32 + 8
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="assignments"):
        rows.RowOrder(one.expand(wide), wide // 8, 8)
    with pytest.raises(ValueError, match="assignments"):
        rows.RowOrder(one.expand(8), -2, -4, pos=one.expand(8))
    order = rows.RowOrder(one, 1, 1)
    x = torch.zeros(1, 1, dtype=torch.bfloat16, device="cuda")
    for call in (rows.dispatch, rows.combine):
        with pytest.raises(MoeError):
            call(x.expand(1, wide), order)
    for shape in ((wide, 1), (1, wide)):
        with pytest.raises(MoeError):
            int8.quantize(x.expand(*shape))
    a, s = torch.zeros(8, 16, dtype=torch.int8, device="cuda"), torch.ones(8, device="cuda")
    index = torch.zeros(8, dtype=torch.int32, device="cuda")
    with pytest.raises(MoeError):
        int8.matmul(a, s, a, s, index=index, index_div=2 ** 32 + 2)
    with pytest.raises(MoeError):
        int8.matmul(a, s, a, s, index=one.expand(wide))
    with pytest.raises(MoeError):
        int8.matmul(a[:1].expand(wide, 16), s[:1].expand(wide), a, s)


def test_orders_and_weights_made_elsewhere():
    """An order and weights made in inference mode, a backward pass taken twice,
    recomputation and saved tensors kept on the host: the same gradients."""
    from torch.utils.checkpoint import checkpoint
    from resident_expert_routing_amd import rows
    T, H, k = 30, 88, 4
    g = torch.Generator().manual_seed(3)
    perm = torch.randperm(T * k, generator=g).int().cuda()
    with torch.inference_mode():
        order = rows.RowOrder(perm.clone(), T, k)
        routed = torch.rand(T, k, generator=g).cuda()
    x = torch.randn(T, H, generator=g).cuda().requires_grad_()
    w = torch.rand(T, k, generator=g).cuda().requires_grad_()
    go = torch.randn(T, H, generator=g).cuda()

    def layer(x, w):
        return rows.combine(rows.dispatch(x, order, routed).tanh(), order, w)

    out = layer(x, w)
    want = torch.autograd.grad(out, [x, w], go, retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(out, [x, w], go), want))
    again = torch.autograd.grad(checkpoint(layer, x, w, use_reentrant=False), [x, w], go)
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    with torch.autograd.graph.save_on_cpu(pin_memory=False):
        out = layer(x, w)
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(out, [x, w], go), want))
    # the formula, in float64: each token's row goes to k places and comes back
    xd, wd = x.detach().cpu().double().requires_grad_(), w.detach().cpu().double().requires_grad_()
    r = routed.cpu().double()
    ref = ((xd.unsqueeze(1) * r.unsqueeze(2)).tanh() * wd.unsqueeze(2)).sum(1)
    for a, b in zip(want, torch.autograd.grad(ref, [xd, wd], go.cpu().double())):
        # a dozen float32 roundings and tanh's few units, sums of at most 88 terms
        assert float((a.cpu().double() - b).norm()) <= 128 * 2.0 ** -24 * 8 * float(b.norm())
