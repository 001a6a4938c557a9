// Products of ragged groups of rows in floating point: the entry points
// moe_grouped_matmul, moe_grouped_outer and moe_swiglu_backward.  The tiled kernels
// are in grouped.hpp.
#include "grouped.hpp"

using namespace moe;

namespace moe {
extern template int launch_rows_product<Bf16>(const RowsProduct&, bool, bool, hipStream_t);
extern template int launch_rows_product<Fp16>(const RowsProduct&, bool, bool, hipStream_t);
extern template int launch_rows_product<float>(const RowsProduct&, bool, bool, hipStream_t);
extern template int launch_outer_product<Bf16>(const OuterProduct&, hipStream_t);
extern template int launch_outer_product<Fp16>(const OuterProduct&, hipStream_t);
extern template int launch_outer_product<float>(const OuterProduct&, hipStream_t);
}  // namespace moe

namespace {

constexpr int kMaxWide = 1 << 24;  // columns, and contraction of a product
constexpr int kMaxRows = 1 << 30;

// The gradient of silu(g) * u:
//   dg = d * u * (s + v * (1 - s)),  du = d * v,  s = 1 / (1 + exp(-g)), v = g * s
// s from exp(-|g|), which cannot overflow.  Below kLow, where 1 - s is 1 in float32, exp(g)
// is applied as two factors exp(g / 2), so that a gradient that is still a normal number
// keeps its value to g = -174: d * u meets them first, or where float32 does not hold it
// (then both are above 1) each of d and u one of them.  Bound by memory (32768 rows of 2048
// bf16, 0.94 GB: 147 us).
// The result is rounded to the element type, since both gradients' products take it as an
// operand of the matrix instruction: with their own rounding the gradients of a bf16 step are
// off by 2.35e-3 of the norm, without it by 1.66e-3 (float32 torch); two parts of 16 bits would
// double both products.  In fp16 values past 65504 are infinite.
template <typename E>
__global__ __launch_bounds__(256) void swiglu_backward_rows(int M, int N, const float* pre,
                                                            size_t pre_stride, const E* dout,
                                                            size_t dout_stride, E* dpre,
                                                            size_t dpre_stride, int chunks,
                                                            int64_t first) {
  constexpr int kN = Piece<E>::kN;
  const int pieces = (N + kN - 1) / kN;
  const int64_t id = first + blockIdx.x;
  const int c = (int)(id % chunks) * 256 + (pieces < 256 ? threadIdx.x % pieces : threadIdx.x);
  const int per = pieces < 256 ? 256 / pieces : 1;
  const int t = pieces < 256 ? threadIdx.x / pieces : 0;
  const int64_t m = id / chunks * per + t;
  if (t >= per || c >= pieces || m >= M) return;
  const int n = c * kN, left = N - n;
  constexpr float kLow = -64.0f;
  Piece<E> d, dg, du;
  float g[kN], u[kN];
  float least = 0.0f;
  const float* z = pre + m * pre_stride + n;
#pragma unroll
  for (int i = 0; i < kN; i += 4) {
    Piece<float> a{}, b{};
    if (left > i) a.load_upto(z + i, left - i), b.load_upto(z + N + i, left - i);
    __builtin_memcpy(g + i, a.e, 16);
    __builtin_memcpy(u + i, b.e, 16);
  }
  d.load_upto(dout + m * dout_stride + n, left);
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const float gf = g[i], uf = u[i], df = to_f32<E>(d.e[i]);
    least = fminf(least, gf);
    const float e = __expf(-fabsf(gf)), near = 1.0f / (1.0f + e), far = e * near;
    const float s = gf < 0.0f ? far : near, rest = gf < 0.0f ? near : far;
    const float v = gf * s;
    dg.e[i] = from_f32<E>(df * uf * fmaf(v, rest, s));
    du.e[i] = from_f32<E>(df * v);
  }
  if (__builtin_expect(least < kLow, 0)) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float gf = g[i], uf = u[i], df = to_f32<E>(d.e[i]);
      const float h = __expf(0.5f * gf);
      if (gf < kLow) {
        const float both = df * uf;
        const float value = fabsf(both) < __builtin_inff() ? (both * h) * ((1.0f + gf) * h)
                                                           : (df * h) * ((uf * h) * (1.0f + gf));
        dg.e[i] = from_f32<E>(value);
        du.e[i] = from_f32<E>((df * h) * (gf * h));
      }
    }
  }
  dg.store_upto(dpre + m * dpre_stride + n, left);
  du.store_upto(dpre + m * dpre_stride + N + n, left);
}

template <typename E>
void launch_swiglu_backward(int M, int N, const float* pre, size_t pre_stride, const void* dout,
                            size_t dout_stride, void* dpre, size_t dpre_stride,
                            hipStream_t stream) {
  const int pieces = (N + Piece<E>::kN - 1) / Piece<E>::kN;
  const int chunks = (pieces + 255) / 256, per = pieces < 256 ? 256 / pieces : 1;
  const int64_t blocks = ((int64_t)M + per - 1) / per * chunks;
  for (int64_t first = 0; first < blocks; first += kMaxGrid) {
    const unsigned grid = (unsigned)(blocks - first < kMaxGrid ? blocks - first : kMaxGrid);
    swiglu_backward_rows<E><<<grid, 256, 0, stream>>>(M, N, pre, pre_stride,
                                                      (const E*)dout, dout_stride, (E*)dpre,
                                                      dpre_stride, chunks, first);
  }
}

int matmul_status(const moe_grouped_matmul_args* a) {
  if (!a) return MOE_EINVAL;
  const size_t e = dtype_bytes(a->dtype), o = dtype_bytes(a->out_dtype);
  if (a->M < 0 || a->N <= 0 || a->K <= 0 || a->G <= 0 || a->a_rows < 0 || e == 0)
    return MOE_EINVAL;
  if (a->out_dtype != a->dtype && a->out_dtype != MOE_DT_FP32) return MOE_EINVAL;
  for (int flag : {a->swiglu, a->b_across, a->zero_rest})
    if (flag != 0 && flag != 1) return MOE_EINVAL;
  if (a->N > kMaxWide || a->K > kMaxWide || a->M > kMaxRows || a->G > MOE_MAX_S)
    return MOE_EUNSUPPORTED;
  if (a->M == 0) return MOE_OK;
  if (!a->a || !a->b || !a->out || !a->offsets || a->a_rows == 0) return MOE_EINVAL;
  if (a->index ? a->index_div < 1 : a->a_rows < a->M) return MOE_EINVAL;
  if (a->pre && !a->swiglu) return MOE_EINVAL;
  if (!aligned(a->pos, 4) || (a->pos && !a->index)) return MOE_EINVAL;
  if (!aligned(a->a, e) || !aligned(a->b, e) || !aligned(a->out, o) || !aligned(a->pre, 4) ||
      !aligned(a->offsets, 4) || !aligned(a->index, 4))
    return MOE_EINVAL;
  const size_t wide = (size_t)a->N * (a->swiglu ? 2 : 1);
  if (a->a_stride < (size_t)a->K || a->out_stride < (size_t)a->N ||
      a->b_stride < (a->b_across ? wide : (size_t)a->K) || (a->pre && a->pre_stride < wide))
    return MOE_EINVAL;
  return MOE_OK;
}

int outer_status(const moe_grouped_outer_args* a) {
  if (!a) return MOE_EINVAL;
  const size_t e = dtype_bytes(a->dtype);
  if (a->M < 0 || a->L <= 0 || a->R <= 0 || a->G <= 0 || a->left_rows < 0 || a->right_rows < 0 ||
      e == 0)
    return MOE_EINVAL;
  if (a->L > kMaxWide || a->R > kMaxWide || a->M > kMaxRows || a->G > MOE_MAX_S)
    return MOE_EUNSUPPORTED;
  if (!a->out || !a->offsets || !aligned(a->out, e) || !aligned(a->offsets, 4)) return MOE_EINVAL;
  if (a->out_stride < (size_t)a->R ||
      (a->G > 1 && a->out_group_stride < (size_t)(a->L - 1) * a->out_stride + (size_t)a->R))
    return MOE_EINVAL;
  const size_t need = moe_grouped_outer_ws_bytes(a->M, a->L, a->R, a->G, a->dtype);
  if (a->ws_bytes < need) return MOE_EWORKSPACE;
  if (need && (!a->ws || !aligned(a->ws, 16))) return MOE_EINVAL;
  if (a->M == 0) return MOE_OK;  // every group is empty: zeros
  if (!a->left || !a->right || !aligned(a->left, e) || !aligned(a->right, e) ||
      !aligned(a->left_index, 4) || !aligned(a->right_index, 4))
    return MOE_EINVAL;
  if (a->left_index && a->right_index) return MOE_EINVAL;
  if (!aligned(a->pos, 4) || (a->pos && !a->left_index && !a->right_index)) return MOE_EINVAL;
  if (a->left_index ? a->left_div < 1 : a->left_rows < a->M) return MOE_EINVAL;
  if (a->right_index ? a->right_div < 1 : a->right_rows < a->M) return MOE_EINVAL;
  if (a->left_stride < (size_t)a->L || a->right_stride < (size_t)a->R) return MOE_EINVAL;
  return MOE_OK;
}

}  // namespace

extern "C" MOE_EXPORT int moe_grouped_matmul(const moe_grouped_matmul_args* a,
                                             hipStream_t stream) {
  const int s = matmul_status(a);
  if (s != MOE_OK || a->M == 0) return s;
  RowsProduct p{};
  p.M = a->M, p.N = a->N, p.K = a->K, p.G = a->G;
  p.a_rows = a->a_rows, p.index_div = a->index_div;
  p.a = a->a, p.b = a->b, p.out = a->out, p.pre = a->pre;
  p.index = a->index, p.pos = a->pos, p.offsets = a->offsets;
  p.a_stride = a->a_stride, p.b_stride = a->b_stride, p.b_group_stride = a->b_group_stride;
  p.out_stride = a->out_stride, p.pre_stride = a->pre_stride;
  p.zero_rest = a->zero_rest;
  p.out_f32 = a->out_dtype == MOE_DT_FP32;
  if (a->dtype == MOE_DT_BF16) return launch_rows_product<Bf16>(p, a->b_across, a->swiglu, stream);
  if (a->dtype == MOE_DT_FP16) return launch_rows_product<Fp16>(p, a->b_across, a->swiglu, stream);
  return launch_rows_product<float>(p, a->b_across, a->swiglu, stream);
}

extern "C" MOE_EXPORT size_t moe_grouped_outer_ws_bytes(int M, int L, int R, int G, int dtype) {
  if (M <= 0 || L <= 0 || R <= 0 || G <= 0 || dtype_bytes(dtype) == 0) return 0;
  const int splits = outer_splits(M, L, R, G, dtype);
  return splits > 1 ? (size_t)splits * (size_t)G * (size_t)L * (size_t)R * 4 : 0;
}

extern "C" MOE_EXPORT int moe_grouped_outer(const moe_grouped_outer_args* a, hipStream_t stream) {
  const int s = outer_status(a);
  if (s != MOE_OK) return s;
  OuterProduct p{};
  p.M = a->M, p.L = a->L, p.R = a->R, p.G = a->G;
  p.left = a->left, p.right = a->right, p.out = a->out, p.offsets = a->offsets;
  p.left_index = a->left_index, p.right_index = a->right_index, p.pos = a->pos;
  p.left_rows = a->left_rows, p.right_rows = a->right_rows;
  p.left_div = a->left_div, p.right_div = a->right_div;
  p.left_stride = a->left_stride, p.right_stride = a->right_stride;
  p.out_stride = a->out_stride, p.out_group_stride = a->out_group_stride;
  p.splits = a->M > 0 ? outer_splits(a->M, a->L, a->R, a->G, a->dtype) : 1;
  p.sums = p.splits > 1 ? (float*)a->ws : nullptr;
  if (a->dtype == MOE_DT_BF16) return launch_outer_product<Bf16>(p, stream);
  if (a->dtype == MOE_DT_FP16) return launch_outer_product<Fp16>(p, stream);
  return launch_outer_product<float>(p, stream);
}

extern "C" MOE_EXPORT int moe_swiglu_backward(int M, int N, int dtype, const float* pre,
                                              size_t pre_stride, const void* dout,
                                              size_t dout_stride, void* dpre, size_t dpre_stride,
                                              hipStream_t stream) {
  const size_t e = dtype_bytes(dtype);
  if (M < 0 || N <= 0 || e == 0) return MOE_EINVAL;
  if (M > kMaxRows || N > kMaxWide) return MOE_EUNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!pre || !dout || !dpre || !aligned(pre, 4) || !aligned(dout, e) || !aligned(dpre, e))
    return MOE_EINVAL;
  if (pre_stride < 2 * (size_t)N || dpre_stride < 2 * (size_t)N || dout_stride < (size_t)N)
    return MOE_EINVAL;
  if (dtype == MOE_DT_BF16)
    launch_swiglu_backward<Bf16>(M, N, pre, pre_stride, dout, dout_stride, dpre, dpre_stride,
                                 stream);
  else if (dtype == MOE_DT_FP16)
    launch_swiglu_backward<Fp16>(M, N, pre, pre_stride, dout, dout_stride, dpre, dpre_stride,
                                 stream);
  else
    launch_swiglu_backward<float>(M, N, pre, pre_stride, dout, dout_stride, dpre, dpre_stride,
                                  stream);
  return hip_status();
}
