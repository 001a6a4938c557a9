"""Refusals of the grouped and 4-bit entry points, on the CPU: every bad argument gets its
documented code before any HIP call, and the torch functions refuse what they cannot take."""
import pytest
import torch

from resident_expert_routing_amd import binding as B
from resident_expert_routing_amd import grouped, int4

FAKE = 1 << 20  # a non-null, aligned address that is never dereferenced on reject paths
WIDE = 2 ** 32  # sizes that a C int would hold as 0
E, U = B.MOE_EINVAL, B.MOE_EUNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(a=None), E), (dict(b=None), E), (dict(out=None), E), (dict(offsets=None), E),
    (dict(a=FAKE + 1), E), (dict(b=FAKE + 1), E), (dict(out=FAKE + 1), E),
    (dict(dtype=2, a=FAKE + 2), E), (dict(offsets=FAKE + 2), E), (dict(index=FAKE + 2, index_div=1), E),
    (dict(index=FAKE, index_div=0), E), (dict(a_rows=7), E), (dict(a_rows=0, index=FAKE, index_div=1), E),
    (dict(M=-1), E), (dict(N=0), E), (dict(K=0), E), (dict(G=0), E), (dict(dtype=3), E),
    (dict(swiglu=2), E), (dict(b_across=-1), E), (dict(zero_rest=3), E),
    (dict(a_stride=99), E), (dict(b_stride=99), E), (dict(out_stride=63), E),
    (dict(b_across=1, b_stride=63), E), (dict(b_across=1, swiglu=1, b_stride=127), E),
    (dict(pre=FAKE, pre_stride=128), E), (dict(swiglu=1, pre=FAKE, pre_stride=127), E),
    (dict(swiglu=1, pre=FAKE + 2, pre_stride=128), E),
    (dict(out_dtype=1), E), (dict(out_dtype=3), E), (dict(out_dtype=2, out=FAKE + 2), E),
    (dict(N=(1 << 24) + 1, out_stride=1 << 25), U), (dict(K=(1 << 24) + 1, a_stride=1 << 25), U),
    (dict(M=(1 << 30) + 1, a_rows=(1 << 30) + 1), U), (dict(G=8193), U),
    (dict(M=WIDE), U), (dict(N=WIDE + 64), U), (dict(index_div=WIDE), U),
    (dict(M=0, a=None, b=None, out=None, offsets=None, a_rows=0), B.MOE_OK),
])
def test_grouped_matmul_refusals(kw, code):
    a = dict(M=8, N=64, K=100, G=2, dtype=0, swiglu=0, b_across=0, zero_rest=0, a_rows=8, a=FAKE,
             a_stride=100, index=None, index_div=0, offsets=FAKE, b=FAKE, b_stride=100,
             b_group_stride=6400, out=FAKE, out_stride=64)
    assert B.moe_grouped_matmul(**(a | kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(left=None), E), (dict(right=None), E), (dict(out=None), E), (dict(offsets=None), E),
    (dict(left=FAKE + 1), E), (dict(out=FAKE + 1), E), (dict(offsets=FAKE + 1), E),
    (dict(left_index=FAKE, left_div=0), E), (dict(right_index=FAKE + 2, right_div=1), E),
    (dict(left_index=FAKE, left_div=1, right_index=FAKE, right_div=1), E),
    (dict(left_rows=7), E), (dict(right_rows=7), E), (dict(M=-1), E), (dict(L=0), E),
    (dict(R=-2), E), (dict(G=0), E), (dict(dtype=7), E), (dict(left_stride=63), E),
    (dict(right_stride=99), E), (dict(out_stride=99), E), (dict(out_group_stride=6399), E),
    (dict(L=(1 << 24) + 1), U), (dict(R=(1 << 24) + 1), U), (dict(G=8193), U),
    (dict(M=(1 << 30) + 1), U), (dict(L=WIDE), U), (dict(right_div=WIDE), U),
    (dict(M=0, out=None), E),  # zeros are still to be written
    (dict(M=30000, left_rows=30000, right_rows=30000), B.MOE_EWORKSPACE),
    (dict(M=30000, left_rows=30000, right_rows=30000, ws=None, ws_bytes=1 << 30), E),
    (dict(M=30000, left_rows=30000, right_rows=30000, ws=FAKE + 8, ws_bytes=1 << 30), E),
])
def test_grouped_outer_refusals(kw, code):
    a = dict(M=8, L=64, R=100, G=2, dtype=0, left_rows=8, right_rows=8, left=FAKE, left_stride=64,
             left_index=None, left_div=1, right=FAKE, right_stride=100, right_index=None,
             right_div=1, offsets=FAKE, out=FAKE, out_stride=100, out_group_stride=6400)
    assert B.moe_grouped_outer(**(a | kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(pre=None), E), (dict(dout=None), E), (dict(dpre=None), E), (dict(pre=FAKE + 2), E),
    (dict(M=-1), E), (dict(N=0), E), (dict(dtype=3), E), (dict(pre_stride=127), E),
    (dict(dout_stride=63), E), (dict(dpre_stride=100), E), (dict(N=(1 << 24) + 1), U),
    (dict(M=WIDE), U), (dict(M=0, pre=None, dout=None, dpre=None), B.MOE_OK),
])
def test_swiglu_backward_refusals(kw, code):
    a = dict(M=8, N=64, dtype=0, pre=FAKE, pre_stride=128, dout=FAKE, dout_stride=64, dpre=FAKE,
             dpre_stride=128)
    assert B.moe_swiglu_backward(**(a | kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(a=None), E), (dict(codes=None), E), (dict(scale=None), E), (dict(out=None), E),
    (dict(a=FAKE + 1), E), (dict(codes=FAKE + 8), E), (dict(scale=FAKE + 4), E),
    (dict(zero=FAKE + 2), E), (dict(out=FAKE + 1), E), (dict(index=FAKE + 1, index_div=1), E),
    (dict(index=FAKE, index_div=0), E), (dict(G=2), E), (dict(offsets=FAKE), E), (dict(M=-1), E),
    (dict(N=0), E), (dict(K=0), E), (dict(G=-1), E), (dict(a_rows=7), E), (dict(a_dtype=4), E),
    (dict(out_dtype=-1), E), (dict(scale_dtype=2), E), (dict(group=16), E), (dict(group=256), E),
    (dict(swiglu=2), E), (dict(a_stride=99), E), (dict(out_stride=63), E),
    (dict(G=2, offsets=FAKE, codes_group_stride=8), E),
    (dict(G=2, offsets=FAKE, scale_group_stride=2), E),
    (dict(G=2, offsets=FAKE, zero=FAKE, zero_group_stride=3), E),
    (dict(K=(1 << 24) + 1, a_stride=1 << 25), U), (dict(N=(1 << 24) + 1, out_stride=1 << 25), U),
    (dict(M=(1 << 30) + 1, a_rows=(1 << 30) + 1), U), (dict(G=8193, offsets=FAKE), U),
    (dict(M=WIDE), U), (dict(group=WIDE + 64), U),
    (dict(M=0, a=None, codes=None, scale=None, out=None, a_rows=0), B.MOE_OK),
])
def test_int4_matmul_refusals(kw, code):
    a = dict(M=8, N=64, K=100, G=0, swiglu=0, a_rows=8, a=FAKE, a_stride=100, a_dtype=0, index=None,
             index_div=0, offsets=None, group=64, codes=FAKE, codes_group_stride=0, scale=FAKE,
             scale_group_stride=0, scale_dtype=0, zero=None, zero_group_stride=0, out=FAKE,
             out_stride=64, out_dtype=0)
    assert B.moe_int4_matmul(**(a | kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(w=None), E), (dict(codes=None), E), (dict(scale=None), E), (dict(w=FAKE + 1), E),
    (dict(codes=FAKE + 8), E), (dict(scale=FAKE + 4), E), (dict(zero=FAKE + 1), E),
    (dict(N=-1), E), (dict(K=0), E), (dict(w_stride=99), E), (dict(dtype=3), E),
    (dict(scale_dtype=2), E), (dict(group=48), E), (dict(K=(1 << 24) + 1, w_stride=1 << 25), U),
    (dict(N=(1 << 25) + 1), U), (dict(N=WIDE), U),
    (dict(N=0, w=None, codes=None, scale=None), B.MOE_OK),
])
def test_int4_quantize_refusals(kw, code):
    a = dict(w=FAKE, N=8, K=100, w_stride=100, dtype=0, group=128, codes=FAKE, scale=FAKE,
             scale_dtype=0)
    assert B.moe_int4_quantize(**(a | kw)) == code


def test_outer_workspace():
    """Only few small matrices over many rows need one, and it stays small."""
    need = B.moe_grouped_outer_ws_bytes
    assert need(30000, 64, 100, 2, 0) == 29 * 2 * 64 * 100 * 4
    assert need(8, 64, 100, 2, 0) == 0 and need(1 << 20, 4096, 4096, 64, 0) == 0
    assert need(0, 64, 100, 2, 0) == 0 and need(WIDE, 64, 100, 2, 0) == 0
    for L, R, G in ((64, 64, 1), (700, 900, 3), (65, 4000, 2), (1, 1, 500), (512, 512, 7)):
        for dt in range(3):
            assert need(1 << 30, L, R, G, dt) <= 9 << 20


def test_int4_sizes():
    assert B.moe_int4_code_bytes(1, 1) == 1024 and B.moe_int4_code_bytes(17, 129) == 4096
    assert B.moe_int4_scale_count(17, 129, 64) == 2 * 4 * 16
    for bad in ((0, 1), (1, 0), (-1, 5), (1, WIDE), ((1 << 25) + 1, 1), (1, (1 << 24) + 1)):
        assert B.moe_int4_code_bytes(*bad) == 0 and B.moe_int4_scale_count(*bad, 128) == 0
    assert B.moe_int4_scale_count(16, 128, 100) == 0


def test_torch_functions_refuse_host_tensors():
    t, off = torch.zeros(4, 16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        grouped.matmul(t, torch.zeros(1, 8, 16), off)
    with pytest.raises(ValueError, match="GPU"):
        int4.quantize(t)
    with pytest.raises(ValueError, match="GPU"):
        int4.pack(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1))
    with pytest.raises(ValueError, match="GPU"):
        int4.Int4Weight(torch.zeros(1, 1, 16, 64, dtype=torch.uint8), torch.zeros(1, 1, 16), N=4, K=16)
    with pytest.raises(ValueError, match="Int4Weight"):
        int4.matmul(t, t)


def test_layout_of_matrices():
    """Matrices are taken as they lie where an axis is contiguous, and copied otherwise."""
    b = torch.zeros(3, 8, 20)
    assert grouped._matrices(b)[1:] == (False, 20, 160)
    kept, across, down, group = grouped._matrices(b.transpose(1, 2))
    assert kept.data_ptr() == b.data_ptr() and (across, down, group) == (True, 20, 160)
    assert grouped._matrices(b[:1].expand(3, 8, 20))[1:] == (False, 20, 0)
    assert grouped._matrices(b[:, :, :7])[1:] == (False, 20, 160)
    for odd in (b[:, :, ::2], b.permute(1, 2, 0)[:, ::2], b[:, :1].expand(3, 8, 20)):
        assert grouped._matrices(odd)[0].is_contiguous()


@pytest.mark.parametrize("kw,code", [
    (dict(pos=FAKE), E), (dict(pos=FAKE + 2, index=FAKE, index_div=1), E),
    (dict(pos=FAKE + 2, index=FAKE, index_div=1, M=0), B.MOE_OK)])
def test_positions_go_with_an_index(kw, code):
    a = dict(M=8, N=64, K=100, G=2, dtype=0, swiglu=0, b_across=0, zero_rest=0, a_rows=8, a=FAKE,
             a_stride=100, index=None, index_div=0, offsets=FAKE, b=FAKE, b_stride=100,
             b_group_stride=6400, out=FAKE, out_stride=64)
    assert B.moe_grouped_matmul(**(a | kw)) == code
    o = dict(M=8, L=64, R=100, G=2, dtype=0, left_rows=8, right_rows=8, left=FAKE, left_stride=64,
             left_index=None, left_div=1, right=FAKE, right_stride=100, right_index=None,
             right_div=1, offsets=FAKE, out=FAKE, out_stride=100, out_group_stride=6400)
    for side in ("left", "right"):
        as_here = {"pos": "pos", "index": f"{side}_index", "index_div": f"{side}_div"}
        names = {as_here[k]: v for k, v in kw.items() if k != "M"}
        assert B.moe_grouped_outer(**(o | names)) == E
