"""More refusals of the row and 8-bit integer operators, on the CPU."""
import pytest
import torch
from torch.autograd import forward_ad

from resident_expert_routing_amd import binding as B
from resident_expert_routing_amd import rows

FAKE = 1 << 20  # a non-null, aligned address that is never dereferenced on reject paths


def test_no_tangent():
    """A tensor that carries a tangent is found, also as a view; others pass."""
    t = torch.randn(4, 6)
    rows.no_tangent("a call", t, None)
    with forward_ad.dual_level():
        rows.no_tangent("a call", t, None)
        d = forward_ad.make_dual(t, torch.ones_like(t))
        for u in (d, d[1:, 2:4], d.t(), 2 * d):
            with pytest.raises(ValueError, match="tangent"):
                rows.no_tangent("a call", t, u)
            with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
                rows.no_tangent("a call", u)
        rows.no_tangent("a call", d.detach().clone().to(torch.int8))
    rows.no_tangent("a call", t)


WIDE = 2 ** 32  # sizes that a C int would hold as 0, and WIDE + n as n


@pytest.mark.parametrize("kw", [dict(T=WIDE), dict(T=WIDE + 8), dict(T=2 ** 31), dict(k=WIDE + 4),
                                dict(T=-WIDE)])
def test_positions_past_32_bits(kw):
    a = dict(perm=FAKE, T=8, k=4, pos=FAKE) | kw
    assert B.moe_positions(**a) == B.MOE_EUNSUPPORTED


@pytest.mark.parametrize("call", [B.moe_dispatch, B.moe_dispatch_backward, B.moe_combine,
                                  B.moe_combine_backward], ids=lambda f: f.__name__)
@pytest.mark.parametrize("kw", [dict(T=WIDE), dict(H=WIDE + 64, src_stride=WIDE + 64,
                                                   dst_stride=WIDE + 64), dict(k=WIDE + 4)])
def test_rows_past_32_bits(call, kw):
    # T = 0 is valid and does nothing, so a T cut to 0 would have passed unseen
    a = dict(T=0, H=64, k=4, dtype=0, pos=FAKE, src=FAKE, src_stride=64, dst=FAKE, dst_stride=64)
    assert call(**(a | kw)) == B.MOE_EUNSUPPORTED


@pytest.mark.parametrize("kw", [dict(M=WIDE), dict(K=WIDE + 100, x_stride=WIDE + 100,
                                                   q_stride=WIDE + 112)])
def test_quantize_past_32_bits(kw):
    a = dict(x=FAKE, M=0, K=100, x_stride=100, dtype=0, q=FAKE, q_stride=112, scale=FAKE)
    assert B.moe_int8_quantize(**(a | kw)) == B.MOE_EUNSUPPORTED
    assert B.moe_int8_row_bytes(WIDE + 16) == 0


@pytest.mark.parametrize("kw", [dict(M=WIDE), dict(N=WIDE + 64, out_stride=WIDE + 64),
                                dict(K=WIDE + 100, a_stride=WIDE + 112, b_stride=WIDE + 112),
                                dict(G=WIDE), dict(a_rows=WIDE + 8),
                                dict(index=FAKE, index_div=WIDE + 2)])
def test_matmul_past_32_bits(kw):
    a = dict(M=0, N=64, K=100, G=0, swiglu=False, a_rows=8, a=FAKE, a_stride=112, a_scale=FAKE,
             index=None, index_div=0, offsets=None, b=FAKE, b_stride=112, b_group_stride=0,
             b_scale=FAKE, b_scale_group_stride=0, out=FAKE, out_stride=64, out_dtype=0)
    assert B.moe_int8_matmul(**(a | kw)) == B.MOE_EUNSUPPORTED
