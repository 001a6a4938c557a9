"""More refusals of the row and 8-bit integer operators, on the CPU."""
import pytest
import torch
from torch.autograd import forward_ad

from resident_expert_routing_amd import rows


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
