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
// codes share an exponent, so the subtraction costs about two bits of float32; activations
// of 32 bits, whose result would show that, take c - z itself, with more instructions, and so
// do sums of the others that end as no number.
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

// The masks and exponents that widen codes, where one instruction can take both: the
// mask from a scalar register and the exponents from a vector register (as literals they
// take two).
template <bool HALF>
struct Widen {
  uint32_t mask, exponents;
  __device__ __forceinline__ Widen() {
    mask = HALF ? 0x03C003C0u : 0x00780078u;
    exponents = HALF ? 0x4C004C00u : 0x41804180u;
    asm("" : "+s"(mask));
    asm("" : "+v"(exponents));
  }
  // eight codes of a word (code 2j at bit 4j, 2j + 1 at bit 16 + 4j) as 16 + c
  __device__ __forceinline__ i32x4 operator()(uint32_t w) const {
    constexpr int kUp = HALF ? 6 : 3;  // code 0 to the top of the mantissa
    const uint32_t at[4] = {w << kUp, HALF ? w << 2 : w >> 1, HALF ? w >> 2 : w >> 5,
                            HALF ? w >> 6 : w >> 9};
    i32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (int)((at[j] & mask) | exponents);
    return v;
  }
};

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

// Eight activations: loaded as they lie (as whole words: kept as single elements they
// would take a register each), and the operands that the matrix instruction takes of
// them.  float32 ones become three bf16 parts that add up to them exactly.
template <typename E>
struct Acts {
  static constexpr int kWords = 2 * (int)sizeof(E), kParts = sizeof(E) == 4 ? 3 : 1;
  i32x4 raw[kWords / 4];
  __device__ __forceinline__ void load(const E* p) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
      raw[i] = __builtin_bit_cast(i32x4, *(const u32x4*)(p + i * (16 / sizeof(E))));
  }
  __device__ __forceinline__ void load_head(const E* p, int n) {  // n elements, then zeros
    constexpr int kN = Piece<E>::kN;
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      Piece<E> u{};
      if (n > i * kN) u.load_upto(p + i * kN, n - i * kN);
      __builtin_memcpy(&raw[i], u.e, 16);
    }
  }
  __device__ __forceinline__ void parts(i32x4 (&v)[kParts]) const {
    if constexpr (kParts == 1) {
      v[0] = raw[0];
    } else {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __int_as_float(raw[i / 4][i % 4]);
#pragma unroll
      for (int t = 0; t < 3; ++t) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[t][j] = (int)__builtin_amdgcn_perm(__float_as_uint(x[2 * j + 1]),
                                               __float_as_uint(x[2 * j]), 0x07060302u);
#pragma unroll
        for (int i = 0; i < 8 && t < 2; ++i) {
          const float cut = __uint_as_float(__float_as_uint(x[i]) & 0xFFFF0000u);
          x[i] = t == 0 && x[i] == cut ? 0.0f : x[i] - cut;
        }
      }
    }
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

// Eight codes less their zero point: small integers, exact in both types.
template <bool HALF>
__device__ __forceinline__ i32x4 centered(uint32_t w, float zero) {
  i32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float lo = (float)(w >> (4 * j) & 15u) - zero, hi = (float)(w >> (16 + 4 * j) & 15u) - zero;
    if constexpr (HALF)
      v[j] = (int)(from_f32<Fp16>(lo).bits | (uint32_t)from_f32<Fp16>(hi).bits << 16);
    else
      v[j] = (int)__builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
  }
  return v;
}

// One word of each quad's lanes as the words of all four quads in every lane.
__device__ __forceinline__ void spread(uint32_t w, uint32_t (&all)[4]) {
  const auto h = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  const auto lo = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
  all[0] = lo[0], all[1] = lo[1], all[2] = hi[0], all[3] = hi[1];
}

// What a workgroup of WK * WN waves computes: up to 16 * MT rows of one group of `a`
// against 16 * NT rows of weights for each of WN waves (with SwiGLU half of them gate
// rows and half their up rows); WK waves share the tiles along K, each a run of them.
template <int MT_, int NT_, int WK_, int WN_>
struct Form {
  static constexpr int MT = MT_, NT = NT_, WK = WK_, WN = WN_, W = WK * WN;
  static constexpr int kCols = 16 * NT * WN;  // rows of weights
};

// Codes go from memory straight to registers, 1 KB of consecutive bytes a load, kCodesAhead
// tiles before their products, and activations kActsAhead quarters of a tile before
// theirs; a lane loads the scale and zero point of one group of four, its quad's.  The
// waves' sums over K are added through LDS in a fixed order.  QUADS: groups in a tile.
template <typename E, typename F, bool GLU, int QUADS>
__device__ __forceinline__ void int4_tile(const Int4Args& p, const Rows& r, int n0,
                                          f32x4* part) {
  constexpr bool HALF = std::is_same_v<E, Fp16>;
  constexpr bool kExact = sizeof(E) == 4;  // codes less their zero points, no correction
  constexpr int MT = F::MT, NT = F::NT, WK = F::WK;
  constexpr int kRing = 8 / NT, kCodesAhead = kRing - 1;
  constexpr int kActs = 128 / (MT * (int)sizeof(Acts<E>)) > 4 ? 4 : 128 / (MT * (int)sizeof(Acts<E>));
  constexpr int kActsAhead = kActs - 1;
  constexpr int kRun = 4 / QUADS;  // tiles of four groups
  static_assert(kRing >= 2 && kActs >= 2, "rings");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int col = lane & 15, quad = lane >> 4, wn = wave / WK, wk = wave % WK;
  const Widen<HALF> widen;
  const int first = n0 + wn * (GLU ? NT / 2 : NT) * 16;  // the wave's first column of out

  // where lane l reads
  struct Sources {
    const uint8_t* codes[NT];
    const uint16_t* scale[NT];
    const uint8_t* zero[NT];
    const E* arow[MT];
  };
  const bool zeros = p.zero != nullptr;
  auto sources = [&](int l) {
    Sources from;
    const int col = l & 15, quad = l >> 4;
#pragma unroll
    for (int s = 0; s < NT; ++s) {
      const bool up = GLU && s >= NT / 2;
      const int row =
          min(first + 16 * (up ? s - NT / 2 : s) + (up ? p.N : 0) + col, p.rows - 1);
      const size_t block = (size_t)(row / kBlock) * p.chunks;
      from.codes[s] = p.codes + (size_t)r.g * p.codes_group_stride + block * kTileBytes +
                      row % kBlock * (kCodes / 2) + 16 * quad;
      const size_t at = block * QUADS * kBlock + row % kBlock;
      from.scale[s] = p.scale + (size_t)r.g * p.scale_group_stride + at;
      // without zero points any bytes are read in their place, those of the scales
      from.zero[s] = zeros ? p.zero + (size_t)r.g * p.zero_group_stride + at
                           : (const uint8_t*)from.scale[s];
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int src = source_row(p, min(r.lo + 16 * t + col, r.hi - 1));
      from.arow[t] = (const E*)p.a + (size_t)max(src, 0) * p.a_stride + 8 * quad;
    }
    return from;
  };
  const Sources from = sources(lane);
  i32x4 ones;
#pragma unroll
  for (int i = 0; i < 4; ++i) ones[i] = HALF ? 0x3C003C00 : 0x3F803F80;

  struct Side {
    uint16_t s[NT];
    uint8_t z[NT];
  };
  // masks in place of branches, which would cut the loop's loads and products to pieces
  const uint32_t is_bf16 = p.scale_dtype == MOE_DT_BF16 ? ~0u : 0u;
  constexpr uint32_t kOffset = kExact ? 0 : 16;
  const uint32_t given = zeros ? 0xFFu : 0u, offset = zeros ? kOffset : kOffset + 8;
  auto load_codes = [&](const Sources& from, i32x4 (&w)[NT], int c) {
#pragma unroll
    for (int s = 0; s < NT; ++s) w[s] = __builtin_nontemporal_load((const i32x4*)(from.codes[s] + (size_t)c * kTileBytes));
  };
  auto load_side = [&](const Sources& from, Side& w, int group) {  // of groups group .. + 3
    const size_t at = (size_t)min(group + quad, p.chunks * QUADS - 1) * kBlock;
#pragma unroll
    for (int s = 0; s < NT; ++s) w.s[s] = from.scale[s][at], w.z[s] = from.zero[s][at];
  };
  f32x4 acc[MT][NT] = {}, dot[MT][NT], sum[MT];
  // products of quarter j of a tile; the first of a group of weights starts its sums
  auto multiply = [&](const uint32_t (&word)[NT][4], const uint32_t (&side)[NT][4], int q, int j,
                      const Acts<E> (&x)[MT]) {
    const bool fresh = j % (4 / QUADS) == 0;
    i32x4 wide[NT];
#pragma unroll
    for (int s = 0; s < NT; ++s)
      wide[s] = kExact ? centered<HALF>(word[s][j], (float)(side[s][q] >> 16)) : widen(word[s][j]);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      i32x4 v[Acts<E>::kParts];
      x[t].parts(v);
#pragma unroll
      for (int u = 0; u < Acts<E>::kParts; ++u) {
        if constexpr (!kExact) sum[t] = mma<HALF>(v[u], ones, fresh && u == 0 ? f32x4{} : sum[t]);
#pragma unroll
        for (int s = 0; s < NT; ++s)
          dot[t][s] = mma<HALF>(v[u], wide[s], fresh && u == 0 ? f32x4{} : dot[t][s]);
      }
    }
  };
  auto scale_of = [&](uint32_t side) {
    const uint32_t bits = side & 0xFFFFu;
    const float half = to_f32<Fp16>(Fp16{(uint16_t)bits});
    return __uint_as_float((bits << 16 & is_bf16) | (__float_as_uint(half) & ~is_bf16));
  };
  auto finish = [&](const uint32_t (&side)[NT][4], int q) {  // a group's sums
#pragma unroll
    for (int s = 0; s < NT; ++s) {
      const float sc = scale_of(side[s][q]);
      const float off = (float)(side[s][q] >> 16);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[t][s][i] = fmaf(sc, kExact ? dot[t][s][i] : fmaf(-off, sum[t][i], dot[t][s][i]),
                              acc[t][s][i]);
    }
  };
  auto spread_side = [&](const Side& w, uint32_t (&side)[NT][4]) {
#pragma unroll
    for (int s = 0; s < NT; ++s)
      spread((uint32_t)w.s[s] | ((w.z[s] & given) + offset) << 16, side[s]);
  };
  auto words = [&](const i32x4 (&w)[NT], uint32_t (&word)[NT][4]) {
#pragma unroll
    for (int s = 0; s < NT; ++s) {
      __builtin_memcpy(word[s], &w[s], 16);
      exchange(word[s]);
    }
  };

  // The wave's whole tiles [lo, hi).  Loads past its last repeat that one, so that nothing
  // branches between loads and products.
  const int full = p.K / kCodes;
  const int lo = (int)((int64_t)full * wk / WK), hi = (int)((int64_t)full * (wk + 1) / WK);
  if (lo < hi) {
    i32x4 w[kRing][NT];
    Acts<E> x[kActs][MT];
    Side next;
    const int last = 4 * (hi - lo) - 1;  // quarter of a tile
    auto load_acts = [&](Acts<E> (&to)[MT], int step) {
      const int k = lo * kCodes + 32 * min(step, last);
#pragma unroll
      for (int t = 0; t < MT; ++t) to[t].load(from.arow[t] + k);
    };
#pragma unroll
    for (int u = 0; u < kCodesAhead; ++u) load_codes(from, w[u], min(lo + u, hi - 1));
    load_side(from, next, lo * QUADS);
#pragma unroll
    for (int u = 0; u < kActsAhead; ++u) load_acts(x[u], u);
    for (int c0 = lo; c0 < hi; c0 += 4) {
      uint32_t side[NT][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = c0 + u;
        if (c >= hi) break;
        load_codes(from, w[(u + kCodesAhead) % kRing], min(c + kCodesAhead, hi - 1));
        if (u % kRun == 0) {
          spread_side(next, side);
          load_side(from, next, (c + kRun) * QUADS);
        }
        uint32_t word[NT][4];
        words(w[u % kRing], word);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          load_acts(x[(4 * u + j + kActsAhead) % kActs], 4 * (c - lo) + j + kActsAhead);
          const int q = (u % kRun) * QUADS + j / (4 / QUADS);
          multiply(word, side, q, j, x[(4 * u + j) % kActs]);
          if ((j + 1) % (4 / QUADS) == 0) finish(side, q);
          __builtin_amdgcn_sched_barrier(0);  // keep to this order: registers
        }
      }
    }
  }
  if (full < p.chunks && wk == WK - 1) {  // the tile that the end of the rows cuts
    i32x4 w[NT];
    Side s;
    uint32_t word[NT][4], side[NT][4];
    load_codes(from, w, full);
    load_side(from, s, full * QUADS);
    words(w, word);
    spread_side(s, side);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = full * kCodes + 32 * j;
      Acts<E> x[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) x[t].load_head(from.arow[t] + k, p.K - k - 8 * quad);
      // a group that begins behind the row has no scale: its weights are padding
      const int q = j / (4 / QUADS);
      multiply(word, side, q, j, x);
      if ((j + 1) % (4 / QUADS) == 0 && full * kCodes + q * (kCodes / QUADS) < p.K)
        finish(side, q);
    }
  }

  // Sums that are no numbers once more, of codes less their zero points: of a * (16 + c) and
  // their correction an infinite activation, or one so large that 31 of it are, makes a NaN
  // where the definition has an infinity or a number.  Other sums keep what they are; those
  // of padding rows, which may hold anything, do not count.
  if constexpr (!kExact) {
    // places and addresses from a copy of the lane's number: kept over the main loop, those
    // from before it cost it a wave a SIMD (one decode step's gate/up 82 us against 73)
    int l = lane;
    asm("" : "+v"(l));
    bool fine = true;
#pragma unroll
    for (int s = 0; s < NT; ++s) {
      const bool padding = first + 16 * (GLU ? s % (NT / 2) : s) + (l & 15) >= p.N;
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          fine = fine && (padding || fabsf(acc[t][s][i]) < __builtin_inff());
    }
    if (__builtin_expect(!__all(fine), 0)) {
      const Sources from = sources(l);
      f32x4 again[MT][NT] = {};
      const int end = wk == WK - 1 ? p.chunks : hi;
#pragma unroll 1
      for (int c = lo; c < end; ++c) {
        i32x4 w[NT];
        Side near;
        uint32_t word[NT][4], side[NT][4];
        load_codes(from, w, c);
        load_side(from, near, c * QUADS);
        words(w, word);
        spread_side(near, side);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = c * kCodes + 32 * j, q = j / (4 / QUADS);
          const bool fresh = j % (4 / QUADS) == 0, last = (j + 1) % (4 / QUADS) == 0;
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            Acts<E> x;
            i32x4 v[1];
            x.load_head(from.arow[t] + k, p.K - k - 8 * quad);
            x.parts(v);
#pragma unroll
            for (int s = 0; s < NT; ++s)
              dot[t][s] = mma<HALF>(v[0], centered<HALF>(word[s][j], (float)(side[s][q] >> 16) - 16.0f),
                                    fresh ? f32x4{} : dot[t][s]);
          }
          if (last && c * kCodes + q * (kCodes / QUADS) < p.K) {
#pragma unroll
            for (int s = 0; s < NT; ++s)
#pragma unroll
              for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  again[t][s][i] = fmaf(scale_of(side[s][q]), dot[t][s][i], again[t][s][i]);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int s = 0; s < NT; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!(fabsf(acc[t][s][i]) < __builtin_inff())) acc[t][s][i] = again[t][s][i];
    }
  }

  // A lane has rows 4 * quad .. + 3 of `a` against row `col` of the weights, and leaves
  // with row `col` of out and columns 4 * quad .. + 3, after the sum over the WK waves.
  const float* sums = (const float*)(part + wn * WK * NT * kWave);
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    if (t) __syncthreads();
#pragma unroll
    for (int s = 0; s < NT; ++s) part[(wave * NT + s) * kWave + lane] = acc[t][s];
    __syncthreads();
    const int m = r.lo + 16 * t + col;
    const bool live = m < r.hi && source_row(p, m) >= 0;
    constexpr int kSets = GLU ? NT / 2 : NT;  // sixteens of columns, dealt to the WK waves
#pragma unroll
    for (int s0 = 0; s0 < kSets; s0 += WK) {
      const int s = s0 + wk, n = first + 16 * s + 4 * quad;
      if (!live || s >= kSets || n >= p.N) continue;
      float y[GLU ? 2 : 1][4] = {};
#pragma unroll
      for (int h = 0; h < (GLU ? 2 : 1); ++h)
#pragma unroll
        for (int k = 0; k < WK; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            y[h][i] += sums[((k * NT + s + h * (NT / 2)) * kWave + col / 4 * 16 + 4 * quad + i) * 4 +
                            col % 4];
      if constexpr (GLU) {
        float h[4];
        swiglu(y[0], y[1], h);
        store_out(p, m, n, h);
      } else {
        store_out(p, m, n, y[0]);
      }
    }
  }
}

template <typename E, typename F, bool GLU, int QUADS>
__global__ __launch_bounds__(F::W* kWave, F::NT == 2 ? 4 : 2) void int4_stream(Int4Args p,
                                                                              int cols,
                                                                              int64_t first) {
  __shared__ f32x4 part[F::W * F::NT * kWave];
  __shared__ int counts[F::W];
  const int64_t w = first + blockIdx.x;
  Rows r;
  if (!find_rows(p, w / cols, 16 * F::MT, counts, r)) return;
  int4_tile<E, F, GLU, QUADS>(p, r, (int)(w % cols) * (GLU ? F::kCols / 2 : F::kCols), part);
}

template <typename F, bool GLU>
int columns(const Int4Args& p) {
  return (p.N + (GLU ? F::kCols / 2 : F::kCols) - 1) / (GLU ? F::kCols / 2 : F::kCols);
}

template <typename E, typename F, bool GLU>
void launch_form(const Int4Args& p, int group, hipStream_t stream) {
  const int cols = columns<F, GLU>(p);
  const int64_t tiles = max_items(p.M, p.G, 16 * F::MT) * cols;
  for (int64_t first = 0; first < tiles; first += kMaxGrid) {
    const unsigned grid = (unsigned)(tiles - first < kMaxGrid ? tiles - first : kMaxGrid);
    if (group == 128)
      int4_stream<E, F, GLU, 1><<<grid, F::W * kWave, 0, stream>>>(p, cols, first);
    else if (group == 64)
      int4_stream<E, F, GLU, 2><<<grid, F::W * kWave, 0, stream>>>(p, cols, first);
    else
      int4_stream<E, F, GLU, 4><<<grid, F::W * kWave, 0, stream>>>(p, cols, first);
  }
}

// Which form.  With few rows in each group the weights bound, and a wave that takes 64 rows
// of them over all of K has the most under way for the least start (one decode step's
// gate/up, 64 rows over 44 groups, 376 MB: 68 us; four waves sharing K, 32 rows of weights
// each, 93; two 87).  That needs enough groups: below kEnough workgroups the waves share K
// (8 groups of one row: 24 us in the first form, 20 with four waves), all eight of them
// where even then CUs would be left without a workgroup (one token, 8.4 MB: 6.1 us).  Groups
// of more rows take tiles of 32, for which weights are widened once (8192 rows over 166
// groups: 790 us against 961; 2048 rows: 501 against 443), where groups and columns alone are
// a workgroup for every CU: tiles of rows are not counted, so dense products and few long
// groups stay at 16 rows.  Tiles of 64 do not fit the registers (1005).
template <typename E, bool GLU>
void launch_matmul(const Int4Args& p, int group, hipStream_t stream) {
  using Few = Form<1, 2, 8, 1>;
  using Mid = Form<1, 2, 4, 1>;
  using Thin = Form<1, 4, 1, 2>;
  using Wide = Form<2, 4, 1, 4>;
  constexpr int kEnough = 640, kCUs = 256;
  const int64_t groups = p.G > 0 ? (p.G < p.M ? p.G : p.M) : 1;
  const bool thin = p.M <= 16 || p.M < 24 * groups;
  if (!thin && groups * columns<Wide, GLU>(p) >= kCUs) {
    launch_form<E, Wide, GLU>(p, group, stream);
  } else if (max_items(p.M, p.G, 16) * columns<Mid, GLU>(p) <= kCUs) {
    launch_form<E, Few, GLU>(p, group, stream);
  } else if (max_items(p.M, p.G, 16) * columns<Thin, GLU>(p) < kEnough) {
    launch_form<E, Mid, GLU>(p, group, stream);
  } else {
    launch_form<E, Thin, GLU>(p, group, stream);
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
  float want = zero ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f;
  if (!(want < __builtin_inff())) want = (0.5f * hi - 0.5f * lo) / 7.5f;  // hi - lo overflowed
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
