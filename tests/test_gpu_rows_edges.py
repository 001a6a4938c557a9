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
