// Products with 4-bit weights and a scale for each group of weights:
// moe_int4_quantize, moe_int4_matmul.
//
//   y[p,n] = sum_q s[g,n,q] * sum_{i in q} a[r,i] * (c[g,n,i] - z[g,n,q])
//
// A code c becomes 16 + c in the matrix instruction's 16-bit type, exactly, by one shift
// and one and-or for two of them; the inner sums are then
//   sum_i a[r,i] * (16 + c[i])  -  (16 + z) * sum_i a[r,i]
// with the second sum from the same instruction against ones, and only finished group
// sums meet the scales, all in float32.  16 is the smallest offset that lets all sixteen
// codes share an exponent, so the subtraction costs about two bits of float32.
#include <type_traits>

#include "groups.hpp"

using namespace moe;

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxWide = 1 << 24;
constexpr int kMaxRows = 1 << 30;
constexpr int kBlock = 16;    // rows of a tile of codes
constexpr int kCodes = 128;   // weights of a row in a tile, 64 bytes
constexpr int kTileBytes = kBlock * kCodes / 2;

inline int blocks_of(int N) { return (N + kBlock - 1) / kBlock; }
inline int chunks_of(int K) { return (K + kCodes - 1) / kCodes; }

struct Int4Args {
  int M, N, K, G, a_rows, index_div, out_dtype, scale_dtype;
  int rows, chunks;  // of a group's codes: rows padded to 16, tiles along a row
  const void* a;
  const int32_t *index, *offsets;
  const uint8_t* codes;
  const uint16_t* scale;
  const uint8_t* zero;
  void* out;
  size_t a_stride, codes_group_stride, scale_group_stride, zero_group_stride, out_stride;
};

// Eight codes of a word (code 2j at bit 4j, 2j + 1 at bit 16 + 4j) as 16 + c.
template <bool HALF>
__device__ __forceinline__ i32x4 widen(uint32_t w) {
  i32x4 v;
  if constexpr (HALF) {
    v[0] = (int)((w << 6 & 0x03C003C0u) | 0x4C004C00u);
    v[1] = (int)((w << 2 & 0x03C003C0u) | 0x4C004C00u);
    v[2] = (int)((w >> 2 & 0x03C003C0u) | 0x4C004C00u);
    v[3] = (int)((w >> 6 & 0x03C003C0u) | 0x4C004C00u);
  } else {
    v[0] = (int)((w << 3 & 0x00780078u) | 0x41804180u);
    v[1] = (int)((w >> 1 & 0x00780078u) | 0x41804180u);
    v[2] = (int)((w >> 5 & 0x00780078u) | 0x41804180u);
    v[3] = (int)((w >> 9 & 0x00780078u) | 0x41804180u);
  }
  return v;
}

template <bool HALF>
__device__ __forceinline__ f32x4 mma(i32x4 w, i32x4 x, f32x4 acc) {
  if constexpr (HALF) {
    typedef _Float16 V __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(V, w),
                                                  __builtin_bit_cast(V, x), acc, 0, 0, 0);
  } else {
    typedef __bf16 V __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(V, w),
                                                   __builtin_bit_cast(V, x), acc, 0, 0, 0);
  }
}

// Words of the four lanes (col, quad 0..3) exchanged: word j of quad q for word q of quad
// j.  A lane's 16 bytes are 32 consecutive weights of a row; afterwards its word j is the
// eight weights 32 j + 8 quad, so that one instruction has 32 consecutive weights and
// stays within a group.
__device__ __forceinline__ void exchange(uint32_t (&w)[4]) {
  auto swap32 = [](uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0], b = r[1];
  };
  auto swap16 = [](uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0], b = r[1];
  };
  swap32(w[0], w[2]);
  swap32(w[1], w[3]);
  swap16(w[0], w[1]);
  swap16(w[2], w[3]);
}

// Eight activations as the matrix instruction takes them.  float32 ones become three
// bf16 parts that add up to them exactly.
template <typename E>
struct Acts {
  static constexpr int kParts = 1;
  i32x4 v[1];
  __device__ __forceinline__ void load(const E* p, int n) {
    Piece<E> u;
    u.load_upto(p, n);
    __builtin_memcpy(&v[0], u.e, 16);
  }
};
template <>
struct Acts<float> {
  static constexpr int kParts = 3;
  i32x4 v[3];
  __device__ __forceinline__ void load(const float* p, int n) {
    Piece<float> u[2];
    u[0].load_upto(p, n);
    if (n > 4)
      u[1].load_upto(p + 4, n - 4);
    else
      u[1] = Piece<float>{};
    uint16_t b[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x = u[i / 4].e[i % 4];
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        b[t][i] = from_f32<Bf16>(x).bits;
        x -= bf16_to_f32(b[t][i]);
      }
    }
#pragma unroll
    for (int t = 0; t < 3; ++t) __builtin_memcpy(&v[t], b[t], 16);
  }
};

template <typename E>
__device__ __forceinline__ void store4(const Int4Args& p, int m, int n, const float (&y)[4]) {
  Piece<E, 4> o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.e[i] = from_f32<E>(y[i]);
  o.store_upto((E*)p.out + (size_t)m * p.out_stride + n, p.N - n);
}

__device__ __forceinline__ void store_out(const Int4Args& p, int m, int n, const float (&y)[4]) {
  if (p.out_dtype == MOE_DT_BF16)
    store4<Bf16>(p, m, n, y);
  else if (p.out_dtype == MOE_DT_FP16)
    store4<Fp16>(p, m, n, y);
  else
    store4<float>(p, m, n, y);
}

// A workgroup takes 32 rows of weights (with SwiGLU, 16 gate rows and their 16 up rows)
// and up to 16 * MT rows of one group of `a`, its W waves the tiles along K in turn; the
// waves' sums are added through LDS in a fixed order.  Codes go from memory straight to
// registers, 1 KB of consecutive bytes a load.  QUADS: groups of weights in a tile.
template <typename E, int W, int MT, bool GLU, int QUADS>
__device__ __forceinline__ void int4_tile(const Int4Args& p, const Rows& r, int n0,
                                          f32x4* part) {
  constexpr bool HALF = std::is_same_v<E, Fp16>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x / kWave;
  const int col = lane & 15, quad = lane >> 4;

  const uint8_t* codes[2];
  int at4[2];  // of the lane's four results: the first row, for scales and zero points
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int first = GLU ? n0 + (s ? p.N : 0) : n0 + 16 * s;
    const int row = min(first + col, p.rows - 1);
    codes[s] = p.codes + (size_t)r.g * p.codes_group_stride +
               ((size_t)(row / kBlock) * p.chunks * kBlock + row % kBlock) * (kCodes / 2) +
               16 * quad;
    at4[s] = first + 4 * quad;
  }
  const uint16_t* scale = p.scale + (size_t)r.g * p.scale_group_stride;
  const uint8_t* zero = p.zero ? p.zero + (size_t)r.g * p.zero_group_stride : nullptr;
  const bool four = !GLU || p.N % 4 == 0;  // a lane's four rows lie side by side
  const int groups = p.chunks * QUADS;
  auto place = [&](int row, int q) {  // of a row's scale and zero point of group q
    return ((size_t)(row / kBlock) * groups + q) * kBlock + row % kBlock;
  };
  auto as_scale = [&](uint16_t b) {
    return p.scale_dtype == MOE_DT_BF16 ? bf16_to_f32(b) : to_f32<Fp16>(Fp16{b});
  };

  const E* arow[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int src = source_row(p, min(r.lo + 16 * t + col, r.hi - 1));
    arow[t] = (const E*)p.a + (size_t)max(src, 0) * p.a_stride + 8 * quad;
  }

  i32x4 ones;
#pragma unroll
  for (int i = 0; i < 4; ++i) ones[i] = HALF ? 0x3C003C00 : 0x3F803F80;
  f32x4 acc[MT][2] = {};

  struct Tile {
    i32x4 c[2];
    uint16_t s[2][QUADS][4];
    uint8_t z[2][QUADS][4];
  };
  auto load = [&](Tile& w, int c) {
#pragma unroll
    for (int s = 0; s < 2; ++s) w.c[s] = *(const i32x4*)(codes[s] + (size_t)c * kTileBytes);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int q = 0; q < QUADS; ++q) {
        if (four) {
          const size_t at = place(min(at4[s], p.rows - 4), c * QUADS + q);
          __builtin_memcpy(w.s[s][q], __builtin_assume_aligned(scale + at, 8), 8);
          if (zero) __builtin_memcpy(w.z[s][q], __builtin_assume_aligned(zero + at, 4), 4);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const size_t at = place(min(at4[s] + i, p.rows - 1), c * QUADS + q);
            w.s[s][q][i] = scale[at];
            if (zero) w.z[s][q][i] = zero[at];
          }
        }
      }
  };
  auto multiply = [&](const Tile& w, int c, auto whole) {
    uint32_t word[2][4];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      __builtin_memcpy(word[s], &w.c[s], 16);
      exchange(word[s]);
    }
#pragma unroll
    for (int q = 0; q < QUADS; ++q) {
      // a group behind the row has no scale; its weights are padding
      if (!decltype(whole)::value && c * kCodes + q * (kCodes / QUADS) >= p.K) break;
      f32x4 dot[MT][2] = {}, sum[MT] = {};
#pragma unroll
      for (int j = q * 4 / QUADS; j < (q + 1) * 4 / QUADS; ++j) {
        const int k = c * kCodes + 32 * j;
        i32x4 wide[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) wide[s] = widen<HALF>(word[s][j]);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          Acts<E> x;
          const int n = decltype(whole)::value ? 8 : p.K - k - 8 * quad;
          if (n > 0)
            x.load(arow[t] + k, n);
          else
            x = Acts<E>{};
#pragma unroll
          for (int u = 0; u < Acts<E>::kParts; ++u) {
            sum[t] = mma<HALF>(ones, x.v[u], sum[t]);
#pragma unroll
            for (int s = 0; s < 2; ++s) dot[t][s] = mma<HALF>(wide[s], x.v[u], dot[t][s]);
          }
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float sc = as_scale(w.s[s][q][i]);
          const float off = zero ? 16.0f + (float)w.z[s][q][i] : 24.0f;
#pragma unroll
          for (int t = 0; t < MT; ++t)
            acc[t][s][i] = fmaf(sc, fmaf(-off, sum[t][i], dot[t][s][i]), acc[t][s][i]);
        }
    }
  };
  constexpr int U = 2;  // tiles of a wave under way
  const int full = p.K / kCodes;
  int c = wave;
  for (; c + W * (U - 1) < full; c += W * U) {
    Tile w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) load(w[u], c + W * u);
#pragma unroll
    for (int u = 0; u < U; ++u) multiply(w[u], c + W * u, std::true_type{});
  }
  for (; c < p.chunks; c += W) {
    Tile w;
    load(w, c);
    multiply(w, c, std::false_type{});
  }

#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int s = 0; s < 2; ++s) part[(wave * MT * 2 + t * 2 + s) * kWave + lane] = acc[t][s];
  __syncthreads();
  for (int t = wave; t < MT; t += W) {
    f32x4 sum[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      sum[s] = part[(t * 2 + s) * kWave + lane];
#pragma unroll
      for (int w = 1; w < W; ++w) sum[s] += part[(w * MT * 2 + t * 2 + s) * kWave + lane];
    }
    // lane: row `col` of out, columns 4 * quad .. + 3 of each 16
    const int m = r.lo + 16 * t + col;
    if (m >= r.hi || source_row(p, m) < 0) continue;
    float y[2][4];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) y[s][i] = sum[s][i];
    const int n = n0 + 4 * quad;
    if (GLU) {
      float h[4];
      swiglu(y[0], y[1], h);
      if (n < p.N) store_out(p, m, n, h);
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (n + 16 * s < p.N) store_out(p, m, n + 16 * s, y[s]);
    }
  }
}

template <typename E, int W, int MT, bool GLU, int QUADS>
__global__ __launch_bounds__(W* kWave) void int4_stream(Int4Args p, int cols, int64_t first) {
  __shared__ f32x4 part[W * MT * 2 * kWave];
  __shared__ int counts[W];
  const int64_t w = first + blockIdx.x;
  Rows r;
  if (!find_rows(p, w / cols, 16 * MT, counts, r)) return;
  const int n0 = (int)(w % cols) * (GLU ? 16 : 32), rows = r.hi - r.lo;
  if (MT == 1 || rows <= 16)
    int4_tile<E, W, 1, GLU, QUADS>(p, r, n0, part);
  else if (MT == 2 || rows <= 32)
    int4_tile<E, W, 2, GLU, QUADS>(p, r, n0, part);
  else
    int4_tile<E, W, MT, GLU, QUADS>(p, r, n0, part);
}

template <typename E, int W, int MT, bool GLU>
void launch_of(const Int4Args& p, int group, int cols, int64_t tiles, hipStream_t stream) {
  for (int64_t first = 0; first < tiles; first += kMaxGrid) {
    const unsigned grid = (unsigned)(tiles - first < kMaxGrid ? tiles - first : kMaxGrid);
    if (group == 128)
      int4_stream<E, W, MT, GLU, 1><<<grid, W * kWave, 0, stream>>>(p, cols, first);
    else if (group == 64)
      int4_stream<E, W, MT, GLU, 2><<<grid, W * kWave, 0, stream>>>(p, cols, first);
    else
      int4_stream<E, W, MT, GLU, 4><<<grid, W * kWave, 0, stream>>>(p, cols, first);
  }
}

template <typename E, bool GLU>
void launch_matmul(const Int4Args& p, int group, hipStream_t stream) {
  const int per = GLU ? 16 : 32, cols = (p.N + per - 1) / per;
  const int64_t groups = p.G > 0 ? (p.G < p.M ? p.G : p.M) : 1;
  if (p.M <= 16 || p.M < 4 * groups) {
    const int64_t tiles = max_items(p.M, p.G, 16) * cols;
    if (tiles <= 512)
      launch_of<E, 8, 1, GLU>(p, group, cols, tiles, stream);
    else
      launch_of<E, 4, 1, GLU>(p, group, cols, tiles, stream);
  } else {
    launch_of<E, 4, 4, GLU>(p, group, cols, max_items(p.M, p.G, 64) * cols, stream);
  }
}

// ---------------------------------------------------------------------------
// moe_int4_quantize
// ---------------------------------------------------------------------------
// A wave takes a tile: lane 4 x + y has 32 consecutive weights of row x.  Weights behind
// the row's end count as zeros, padding rows get codes and zero points of 8 and scale 0.
template <typename E>
__global__ __launch_bounds__(kWave) void quantize_tiles(const E* w, int N, int K, size_t stride,
                                                        int chunks, int lanes, uint8_t* codes,
                                                        uint16_t* scale, int scale_dtype,
                                                        uint8_t* zero, int64_t first) {
  const int64_t id = first + blockIdx.x;
  const int block = (int)(id / chunks), c = (int)(id % chunks);
  const int lane = threadIdx.x, x = lane >> 2, y = lane & 3;
  const int n = block * kBlock + x, k = c * kCodes + 32 * y;
  constexpr int kN = Piece<E>::kN;
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; i += kN) {
    Piece<E> u{};
    if (n < N && k + i < K) u.load_upto(w + (size_t)n * stride + k + i, K - k - i);
#pragma unroll
    for (int e = 0; e < kN; ++e) v[i + e] = to_f32<E>(u.e[e]);
  }
  float lo = 0.0f, hi = 0.0f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    lo = fminf(lo, v[i]), hi = fmaxf(hi, v[i]);
    finite = finite && fabsf(v[i]) < __builtin_inff();
  }
  int bad = !finite;
  for (int d = 1; d < lanes; d <<= 1) {
    lo = fminf(lo, __shfl_xor(lo, d, 64)), hi = fmaxf(hi, __shfl_xor(hi, d, 64));
    bad |= __shfl_xor(bad, d, 64);
  }
  const float want = zero ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f;
  uint16_t bits = scale_dtype == MOE_DT_BF16 ? from_f32<Bf16>(want).bits : from_f32<Fp16>(want).bits;
  float s = scale_dtype == MOE_DT_BF16 ? bf16_to_f32(bits) : to_f32<Fp16>(Fp16{bits});
  if (bad || !(s < __builtin_inff())) {
    bits = scale_dtype == MOE_DT_BF16 ? 0x7FC0 : 0x7E00;  // NaN
    s = 0.0f;
  }
  const float z = !zero ? 8.0f : s > 0.0f ? fminf(__builtin_rintf(-lo / s), 15.0f) : 8.0f;
  uint32_t word[4] = {};
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float q = s > 0.0f ? __builtin_rintf(v[i] / s) : 0.0f;
    const uint32_t code = (uint32_t)fminf(fmaxf(q + z, 0.0f), 15.0f);
    word[i / 8] |= code << (4 * (i % 8 / 2) + 16 * (i % 2));
  }
  uint8_t* to = codes + ((size_t)id * kBlock + x) * (kCodes / 2) + 16 * y;
  __builtin_memcpy(__builtin_assume_aligned(to, 16), word, 16);
  if (y % lanes == 0) {
    const int per = 4 / lanes;
    const size_t at = ((size_t)block * chunks * per + (size_t)c * per + y / lanes) * kBlock + x;
    scale[at] = bits;
    if (zero) zero[at] = (uint8_t)z;
  }
}

int group_status(int group) {
  return group == 32 || group == 64 || group == 128 ? MOE_OK : MOE_EINVAL;
}

int scale_status(int dtype) {
  return dtype == MOE_DT_BF16 || dtype == MOE_DT_FP16 ? MOE_OK : MOE_EINVAL;
}

int matmul_status(const moe_int4_matmul_args* a) {
  if (!a) return MOE_EINVAL;
  const size_t e = dtype_bytes(a->a_dtype), o = dtype_bytes(a->out_dtype);
  if (a->M < 0 || a->N <= 0 || a->K <= 0 || a->G < 0 || a->a_rows < 0) return MOE_EINVAL;
  if (e == 0 || o == 0 || (a->swiglu != 0 && a->swiglu != 1) || group_status(a->group) != MOE_OK ||
      scale_status(a->scale_dtype) != MOE_OK)
    return MOE_EINVAL;
  if (a->K > kMaxWide || a->N > kMaxWide || a->M > kMaxRows || a->G > MOE_MAX_S)
    return MOE_EUNSUPPORTED;
  if (a->M == 0) return MOE_OK;
  if (!a->a || !a->codes || !a->scale || !a->out || a->a_rows == 0) return MOE_EINVAL;
  if ((a->G > 0) != (a->offsets != nullptr)) return MOE_EINVAL;
  if (a->index ? a->index_div < 1 : a->a_rows < a->M) return MOE_EINVAL;
  if (!aligned(a->a, e) || !aligned(a->out, o) || !aligned(a->codes, 16) ||
      a->codes_group_stride % 16 || !aligned(a->scale, 8) || a->scale_group_stride % 4 ||
      !aligned(a->zero, 4) || a->zero_group_stride % 4 || !aligned(a->index, 4) ||
      !aligned(a->offsets, 4))
    return MOE_EINVAL;
  if (a->a_stride < (size_t)a->K || a->out_stride < (size_t)a->N) return MOE_EINVAL;
  return MOE_OK;
}

}  // namespace

extern "C" MOE_EXPORT size_t moe_int4_code_bytes(int N, int K) {
  if (N <= 0 || K <= 0 || K > kMaxWide || N > 2 * kMaxWide) return 0;
  return (size_t)blocks_of(N) * chunks_of(K) * kTileBytes;
}

extern "C" MOE_EXPORT size_t moe_int4_scale_count(int N, int K, int group) {
  if (N <= 0 || K <= 0 || K > kMaxWide || N > 2 * kMaxWide || group_status(group) != MOE_OK)
    return 0;
  return (size_t)blocks_of(N) * chunks_of(K) * (kCodes / group) * kBlock;
}

extern "C" MOE_EXPORT int moe_int4_quantize(const void* w, int N, int K, size_t w_stride,
                                            int dtype, int group, uint8_t* codes, void* scale,
                                            int scale_dtype, uint8_t* zero, hipStream_t stream) {
  const size_t e = dtype_bytes(dtype);
  if (N < 0 || K <= 0 || e == 0 || group_status(group) != MOE_OK ||
      scale_status(scale_dtype) != MOE_OK)
    return MOE_EINVAL;
  if (K > kMaxWide || N > 2 * kMaxWide) return MOE_EUNSUPPORTED;
  if (N == 0) return MOE_OK;
  if (!w || !codes || !scale || !aligned(w, e) || !aligned(codes, 16) || !aligned(scale, 8) ||
      !aligned(zero, 4) || w_stride < (size_t)K)
    return MOE_EINVAL;
  const int chunks = chunks_of(K), lanes = group / 32;
  const int64_t tiles = (int64_t)blocks_of(N) * chunks;
  for (int64_t first = 0; first < tiles; first += kMaxGrid) {
    const unsigned grid = (unsigned)(tiles - first < kMaxGrid ? tiles - first : kMaxGrid);
    if (dtype == MOE_DT_BF16)
      quantize_tiles<Bf16><<<grid, kWave, 0, stream>>>((const Bf16*)w, N, K, w_stride, chunks, lanes,
                                                       codes, (uint16_t*)scale, scale_dtype, zero,
                                                       first);
    else if (dtype == MOE_DT_FP16)
      quantize_tiles<Fp16><<<grid, kWave, 0, stream>>>((const Fp16*)w, N, K, w_stride, chunks, lanes,
                                                       codes, (uint16_t*)scale, scale_dtype, zero,
                                                       first);
    else
      quantize_tiles<float><<<grid, kWave, 0, stream>>>((const float*)w, N, K, w_stride, chunks,
                                                        lanes, codes, (uint16_t*)scale, scale_dtype,
                                                        zero, first);
  }
  return hip_status();
}

extern "C" MOE_EXPORT int moe_int4_matmul(const moe_int4_matmul_args* a, hipStream_t stream) {
  const int s = matmul_status(a);
  if (s != MOE_OK || a->M == 0) return s;
  Int4Args p{};
  p.M = a->M, p.N = a->N, p.K = a->K, p.G = a->G;
  p.a_rows = a->a_rows, p.index_div = a->index_div;
  p.out_dtype = a->out_dtype, p.scale_dtype = a->scale_dtype;
  p.rows = blocks_of(a->N * (a->swiglu ? 2 : 1)) * kBlock, p.chunks = chunks_of(a->K);
  p.a = a->a, p.index = a->index, p.offsets = a->offsets;
  p.codes = a->codes, p.scale = (const uint16_t*)a->scale, p.zero = a->zero, p.out = a->out;
  p.a_stride = a->a_stride, p.out_stride = a->out_stride;
  p.codes_group_stride = a->codes_group_stride, p.scale_group_stride = a->scale_group_stride;
  p.zero_group_stride = a->zero_group_stride;
  auto launch = [&](auto type) {
    using E = decltype(type);
    if (a->swiglu)
      launch_matmul<E, true>(p, a->group, stream);
    else
      launch_matmul<E, false>(p, a->group, stream);
  };
  if (a->a_dtype == MOE_DT_BF16)
    launch(Bf16{});
  else if (a->a_dtype == MOE_DT_FP16)
    launch(Fp16{});
  else
    launch(0.0f);
  return hip_status();
}
