"""Grouped products in floating point against float64 (grouped_oracle has the bounds)."""
import pytest
import torch

from grouped_oracle import Reference, bucketing, within, worst

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32

# rows of the groups, columns of out, K: group sizes on both sides of every tile height,
# sizes that end inside a tile, a stage and a 16-byte piece
SHAPES = [
    ([1], 1, 1),
    ([1, 0, 2], 7, 5),
    ([3, 0, 0, 17, 64], 128, 64),
    ([65, 1, 128, 0], 256, 128),
    ([129, 192, 5], 264, 72),
    ([193, 256, 31], 136, 200),
    ([257, 320, 0, 7], 384, 136),
    ([321, 2, 640], 120, 1032),
    ([66, 130, 300], 257, 259),
    ([40, 0, 333], 33, 515),
    ([0, 0, 0], 64, 64),
]


def inputs(counts, N, K, dtype, swiglu, across, by_token, seed, tail=3):
    gen = torch.Generator().manual_seed(seed)
    perm, offsets = bucketing(counts, gen, tail=tail)
    M, G = perm.numel(), len(counts)
    wide = 2 * N if swiglu else N
    k = 2 if by_token else 1
    if by_token and M % 2:
        perm = torch.cat([perm, torch.full((1,), -1, dtype=torch.int32)])
        M += 1
    rows = M // k if by_token else M
    a = (torch.randn(rows, K, generator=gen) * 0.7).to(dtype)
    b = torch.randn(G, wide, K, generator=gen) * (1.5 * K ** -0.5)
    b = b.transpose(1, 2).contiguous().to(dtype) if across else b.to(dtype)
    d = torch.randn(M, N, generator=gen).to(dtype)
    dev = "cuda"
    b = b.to(dev)
    return (a.to(dev), b, b.transpose(1, 2) if across else b, perm.to(dev), offsets.to(dev),
            d.to(dev), k, M)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("swiglu,across,by_token", [(False, False, False), (True, False, True),
                                                    (False, True, True), (True, True, False)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_products_and_gradients(shape, swiglu, across, by_token, dtype):
    from resident_expert_routing_amd import grouped, rows
    counts, N, K = SHAPES[shape]
    a, store, b, perm, offsets, d, k, M = inputs(counts, N, K, dtype, swiglu, across, by_token,
                                                 shape)
    index = torch.where(perm < 0, perm, perm // k) if by_token else None
    ref = Reference(a, b, offsets, index, M, swiglu, dtype, d, token_sum=by_token)

    kw = dict(index=perm, index_div=k) if by_token else {}
    with torch.no_grad():
        y = grouped.matmul(a, b, offsets, swiglu=swiglu, **kw)
    print(f"forward {worst(y, ref.out, ref.out_tol):.3f}", flush=True)
    assert within(y, ref.out, ref.out_tol)

    a.requires_grad_(), store.requires_grad_()
    b = store.transpose(1, 2) if across else store
    order = rows.RowOrder(perm, M // k, k) if by_token else None
    y2 = grouped.matmul(a, b, offsets, order=order, swiglu=swiglu)
    assert torch.equal(y, y2)
    da, db = torch.autograd.grad(y2, [a, store], d)
    db = db.transpose(1, 2) if across else db
    print(f"da {worst(da, ref.da, ref.da_tol):.3f} db {worst(db, ref.db, ref.db_tol):.3f}",
          flush=True)
    assert within(da, ref.da, ref.da_tol)
    assert within(db, ref.db, ref.db_tol)
