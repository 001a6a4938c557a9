"""Refusals of the row and 8-bit integer entry points, on the CPU: every bad
argument gets its documented code before any HIP call, and the torch functions
refuse what they cannot take."""
import numpy as np
import pytest
import torch

import resident_expert_routing_amd  # noqa: F401
from resident_expert_routing_amd import binding as B
from resident_expert_routing_amd import int8, rows

FAKE = 1 << 20  # a non-null, aligned address that is never dereferenced on reject paths
BIG = 1 << 30


@pytest.mark.parametrize("kw,code", [
    (dict(perm=None), B.MOE_EINVAL),
    (dict(pos=None), B.MOE_EINVAL),
    (dict(perm=FAKE + 2), B.MOE_EINVAL),
    (dict(pos=FAKE + 1), B.MOE_EINVAL),
    (dict(perm_copy=FAKE + 2), B.MOE_EINVAL),
    (dict(T=-1), B.MOE_EINVAL),
    (dict(k=0), B.MOE_EINVAL),
    (dict(k=33), B.MOE_EUNSUPPORTED),
    (dict(T=1 << 30), B.MOE_EUNSUPPORTED),
    (dict(T=0, perm=None, pos=None), B.MOE_OK),
])
def test_positions_refusals(kw, code):
    a = dict(perm=FAKE, T=8, k=4, pos=FAKE) | kw
    assert B.moe_positions(**a) == code


CALLS = {
    "dispatch": (B.moe_dispatch, dict(perm=None), False),
    "dispatch_backward": (B.moe_dispatch_backward, {}, True),
    "combine": (B.moe_combine, {}, False),
    "combine_backward": (B.moe_combine_backward, dict(perm=None), True),
}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("kw,code", [
    (dict(pos=None), B.MOE_EINVAL),
    (dict(src=None), B.MOE_EINVAL),
    (dict(dst=None), B.MOE_EINVAL),
    (dict(pos=FAKE + 2), B.MOE_EINVAL),
    (dict(src=FAKE + 1), B.MOE_EINVAL),
    (dict(dst=FAKE + 1), B.MOE_EINVAL),
    (dict(dtype=2, src=FAKE + 2), B.MOE_EINVAL),
    (dict(weight=FAKE + 2), B.MOE_EINVAL),
    (dict(T=-1), B.MOE_EINVAL),
    (dict(H=0), B.MOE_EINVAL),
    (dict(H=-5), B.MOE_EINVAL),
    (dict(k=0), B.MOE_EINVAL),
    (dict(dtype=3), B.MOE_EINVAL),
    (dict(dtype=-1), B.MOE_EINVAL),
    (dict(src_stride=63), B.MOE_EINVAL),
    (dict(dst_stride=0), B.MOE_EINVAL),
    (dict(k=33), B.MOE_EUNSUPPORTED),
    (dict(T=1 << 29), B.MOE_EUNSUPPORTED),
    (dict(H=BIG + 1, src_stride=BIG + 1, dst_stride=BIG + 1), B.MOE_EUNSUPPORTED),
    (dict(T=0, pos=None, src=None, dst=None), B.MOE_OK),
])
def test_rows_refusals(name, kw, code):
    call, extra, _ = CALLS[name]
    a = dict(T=8, H=64, k=4, dtype=0, pos=FAKE, src=FAKE, src_stride=64, dst=FAKE, dst_stride=64)
    assert call(**(a | extra | kw)) == code


@pytest.mark.parametrize("name", [n for n in sorted(CALLS) if CALLS[n][2]])
@pytest.mark.parametrize("kw", [
    dict(dweight=FAKE),                                        # no forward input
    dict(other=FAKE, other_stride=64),                         # nothing to compute with it
    dict(dweight=FAKE, other=FAKE, other_stride=63),
    dict(dweight=FAKE + 1, other=FAKE, other_stride=64),
    dict(dweight=FAKE, other=FAKE + 1, other_stride=64),
])
def test_rows_backward_refusals(name, kw):
    a = dict(T=8, H=64, k=4, dtype=0, pos=FAKE, src=FAKE, src_stride=64, dst=FAKE, dst_stride=64)
    assert CALLS[name][0](**(a | kw)) == B.MOE_EINVAL


def test_rows_arguments_of_the_other_calls():
    """perm belongs to the calls that write rows, dweight and other to the backward calls."""
    import ctypes
    lib = B.load()
    base = dict(T=8, H=64, k=4, dtype=0, pos=FAKE, src=FAKE, src_stride=64, dst=FAKE,
                dst_stride=64, weight=None)
    for fn, kw in ((lib.moe_combine, dict(perm=FAKE)), (lib.moe_dispatch_backward, dict(perm=FAKE)),
                   (lib.moe_combine, dict(dweight=FAKE, other=FAKE, other_stride=64)),
                   (lib.moe_dispatch, dict(dweight=FAKE, other=FAKE, other_stride=64))):
        assert fn(B._rows_args(**(base | kw)), None) == B.MOE_EINVAL
    for fn in (lib.moe_combine, lib.moe_combine_backward, lib.moe_dispatch,
               lib.moe_dispatch_backward, lib.moe_int8_matmul):
        null = ctypes.POINTER(B.RowsArgs if fn is not lib.moe_int8_matmul else B.Int8MatmulArgs)()
        assert fn(null, None) == B.MOE_EINVAL


def test_int8_row_bytes():
    assert [B.moe_int8_row_bytes(k) for k in (1, 15, 16, 17, 4096, 131056)] == \
        [16, 16, 16, 32, 4096, 131056]
    assert [B.moe_int8_row_bytes(k) for k in (0, -1, 131057)] == [0, 0, 0]


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), B.MOE_EINVAL),
    (dict(q=None), B.MOE_EINVAL),
    (dict(scale=None), B.MOE_EINVAL),
    (dict(x=FAKE + 1), B.MOE_EINVAL),
    (dict(q=FAKE + 8), B.MOE_EINVAL),
    (dict(scale=FAKE + 2), B.MOE_EINVAL),
    (dict(M=-1), B.MOE_EINVAL),
    (dict(K=0), B.MOE_EINVAL),
    (dict(x_stride=99), B.MOE_EINVAL),
    (dict(q_stride=100), B.MOE_EINVAL),
    (dict(q_stride=96), B.MOE_EINVAL),
    (dict(dtype=3), B.MOE_EINVAL),
    (dict(K=131057, x_stride=131057, q_stride=1 << 18), B.MOE_EUNSUPPORTED),
    (dict(M=0, x=None, q=None, scale=None), B.MOE_OK),
])
def test_quantize_refusals(kw, code):
    a = dict(x=FAKE, M=4, K=100, x_stride=100, dtype=0, q=FAKE, q_stride=112, scale=FAKE)
    assert B.moe_int8_quantize(**(a | kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(a=None), B.MOE_EINVAL),
    (dict(b=None), B.MOE_EINVAL),
    (dict(a_scale=None), B.MOE_EINVAL),
    (dict(b_scale=None), B.MOE_EINVAL),
    (dict(out=None), B.MOE_EINVAL),
    (dict(a=FAKE + 8), B.MOE_EINVAL),
    (dict(b=FAKE + 4), B.MOE_EINVAL),
    (dict(out=FAKE + 1), B.MOE_EINVAL),
    (dict(out_dtype=2, out=FAKE + 2), B.MOE_EINVAL),
    (dict(a_scale=FAKE + 1), B.MOE_EINVAL),
    (dict(index=FAKE + 1, index_div=1), B.MOE_EINVAL),
    (dict(index=FAKE, index_div=0), B.MOE_EINVAL),
    (dict(M=-1), B.MOE_EINVAL),
    (dict(N=0), B.MOE_EINVAL),
    (dict(K=0), B.MOE_EINVAL),
    (dict(G=-1), B.MOE_EINVAL),
    (dict(G=2), B.MOE_EINVAL),                       # groups without offsets
    (dict(offsets=FAKE), B.MOE_EINVAL),              # offsets without groups
    (dict(a_rows=7), B.MOE_EINVAL),
    (dict(a_rows=0, index=FAKE, index_div=1), B.MOE_EINVAL),
    (dict(out_dtype=5), B.MOE_EINVAL),
    (dict(a_stride=100), B.MOE_EINVAL),
    (dict(a_stride=96), B.MOE_EINVAL),
    (dict(b_stride=96), B.MOE_EINVAL),
    (dict(out_stride=63), B.MOE_EINVAL),
    (dict(G=2, offsets=FAKE, b_group_stride=63 * 112, b_scale_group_stride=64), B.MOE_EINVAL),
    (dict(G=2, offsets=FAKE, b_group_stride=64 * 112, b_scale_group_stride=63), B.MOE_EINVAL),
    (dict(G=2, offsets=FAKE, b_group_stride=64 * 112 + 8, b_scale_group_stride=64), B.MOE_EINVAL),
    (dict(G=9000, offsets=FAKE, b_group_stride=64 * 112, b_scale_group_stride=64),
     B.MOE_EUNSUPPORTED),
    (dict(K=131057, a_stride=1 << 18, b_stride=1 << 18), B.MOE_EUNSUPPORTED),
    (dict(N=(1 << 24) + 1, out_stride=1 << 25), B.MOE_EUNSUPPORTED),
    (dict(M=(1 << 30) + 1, a_rows=(1 << 30) + 1), B.MOE_EUNSUPPORTED),
    (dict(M=0, a=None, b=None, a_scale=None, b_scale=None, out=None, a_rows=0), B.MOE_OK),
])
def test_matmul_refusals(kw, code):
    a = dict(M=8, N=64, K=100, G=0, swiglu=False, a_rows=8, a=FAKE, a_stride=112, a_scale=FAKE,
             index=None, index_div=0, offsets=None, b=FAKE, b_stride=112, b_group_stride=0,
             b_scale=FAKE, b_scale_group_stride=0, out=FAKE, out_stride=64, out_dtype=0)
    assert B.moe_int8_matmul(**(a | kw)) == code


def test_torch_functions_refuse_host_tensors():
    perm = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        rows.RowOrder(perm, 4, 2)
    with pytest.raises(ValueError, match="GPU"):
        int8.quantize(torch.zeros(4, 16))
    q = torch.zeros(4, 16, dtype=torch.int8)
    with pytest.raises(ValueError, match="GPU"):
        int8.matmul(q, torch.ones(4), q, torch.ones(4))


def test_pad_rows_layout():
    """pad_rows lays rows out at multiples of 16 bytes and keeps what already is."""
    for shape in ((3, 16), (3, 17), (2, 5, 33), (1, 1, 7), (4, 1)):
        q = torch.from_numpy(np.arange(np.prod(shape)).astype(np.int8).reshape(shape))
        p = int8.pad_rows(q)
        assert torch.equal(p, q) and int8._laid_out(p)
        assert p.stride(-2) % 16 == 0 or p.shape[-2] == 1
        assert int8.pad_rows(p) is p
    t = torch.zeros(32, 64, dtype=torch.int8)
    assert int8.pad_rows(t.t()).is_contiguous()      # transposed: copied
    assert int8.pad_rows(t[:, 16:48]).data_ptr() == t.data_ptr() + 16
    assert int8.pad_rows(t[:, 8:40]).data_ptr() != t.data_ptr() + 8
    assert not int8._laid_out(torch.zeros(1, 64, dtype=torch.int8).expand(4, 64))
