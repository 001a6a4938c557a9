// 8-bit integer rows and their matrix products: moe_int8_quantize,
// moe_int8_matmul.
//
//   s[m]   = max(max_i |x[m,i]| / 127, 2^-126),  q[m,i] = round(x[m,i] / s[m])
//   y[p,n] = sa[r] * sb[g,n] * sum_i qa[r,i] * qb[g,n,i]
//
// The sums are exact 32-bit integers on the matrix cores, so neither the order
// of the contraction nor how it is split over waves changes a result; the two
// scales are applied to the finished sum in float32.
//
// Two times "A against B" in a comment are of one form against the other on one
// card when that choice was made; the times at the head of a kernel's comment are
// the present ones.
#include <type_traits>

#include "groups.hpp"

using namespace moe;

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr float kMinScale = 1.17549435e-38f;  // 2^-126, the smallest normal float
constexpr int kMaxK = 131056;                 // 128 * 128 * K stays below 2^31

__host__ __device__ inline int up16(int v) { return (v + 15) & ~15; }

// ---------------------------------------------------------------------------
// moe_int8_quantize
// ---------------------------------------------------------------------------
constexpr int kQThreads = 256;
constexpr int kQPieces = 4;  // 16-byte pieces of a row that a thread keeps

// round(x / s) to the nearest integer, ties to even, of the exact quotient, for
// a quotient that x * (1 / s) puts next to a half: the candidate q is decided by
// the remainder x - q*s, exact in float64.
__device__ __forceinline__ int settled(float x, float s, int q) {
  const double e = fma(-(double)q, (double)s, (double)x), half = 0.5 * (double)s;
  if (fabs(e) > half || (fabs(e) == half && (q & 1))) q += e > 0 ? 1 : -1;
  return q;
}

// N quotients as bytes.  x * inv is within 2e-5 of the quotient (|quotient| <=
// 127 and a bit, roundings of 2^-24 each), so its rounding is the quotient's
// unless it lies within 1e-4 of a half, which is rare.  Adding 1.5 * 2^23 rounds
// to an integer, ties to even, and leaves it in the sum's low byte.
template <typename E, int N>
__device__ __forceinline__ void quantize_piece(const Piece<E, N>& u, float s, float inv,
                                               int8_t* out) {
  constexpr float kRound = 12582912.0f;
  uint32_t bits[N];
  float off = 0.0f;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float x = to_f32<E>(u.e[e]), t = fmaf(x, inv, kRound);
    bits[e] = __float_as_uint(t);
    off = fmaxf(off, fabsf(fmaf(x, inv, -(t - kRound))));
  }
  if (__builtin_expect(off > 0.4999f, 0)) {
#pragma unroll
    for (int e = 0; e < N; ++e)
      bits[e] = (uint32_t)settled(to_f32<E>(u.e[e]), s, (int)(int8_t)bits[e]);
  }
  uint32_t w[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint32_t lo = __builtin_amdgcn_perm(bits[4 * i + 1], bits[4 * i], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(bits[4 * i + 3], bits[4 * i + 2], 0x0C0C0400u);
    w[i] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
  }
  __builtin_memcpy(out, w, N);
}

// The largest magnitude of a piece, as the bits of a float.  Types of 16 bits
// compare two at a time; order and NaN are as for the floats they stand for.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
template <typename E, int N>
__device__ __forceinline__ uint32_t top_bits(const Piece<E, N>& u, uint32_t top) {
  uint32_t w[N * sizeof(E) / 4];
  __builtin_memcpy(w, u.e, sizeof(w));
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) top = max(top, w[i] & 0x7FFFFFFFu);
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      top = __builtin_bit_cast(
          uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, top),
                                              __builtin_bit_cast(u16x2, w[i] & 0x7FFF7FFFu)));
  }
  return top;
}
template <typename E>
__device__ __forceinline__ uint32_t as_f32_bits(uint32_t top) {
  if constexpr (sizeof(E) == 4) {
    return top;
  } else {
    const uint32_t m = max(top & 0xFFFFu, top >> 16);
    return __float_as_uint(to_f32<E>(E{(uint16_t)m}));
  }
}

// One pass: the row stays in registers between its maximum and its rounding
// (rows past 256 threads x 4 pieces are read again, from the cache), a wave for a
// row of up to 4 KB, a workgroup for longer ones.  Bound by memory: 65536 rows of
// 2048 bf16 take 72 to 74 us (403 MB, 5.4 to 5.6 TB/s).  A row that holds an
// infinity or a NaN gets scale NaN and zeros, so that everything computed from it
// is NaN.
template <typename E>
__global__ __launch_bounds__(kQThreads) void quantize_rows(const E* __restrict__ x, int M, int K,
                                                           size_t x_stride, int8_t* __restrict__ q,
                                                           size_t q_stride,
                                                           float* __restrict__ scale, int lanes) {
  constexpr int N = Piece<E>::kN;
  __shared__ uint32_t part[kQThreads / kWave];
  const int per = kQThreads / lanes;
  const int lane = threadIdx.x & (lanes - 1);
  const int width = up16(K);
  for (int64_t b = (int64_t)blockIdx.x * per; b < M; b += (int64_t)gridDim.x * per) {
    const int64_t m = b + threadIdx.x / lanes;
    const E* row = x + (m < M ? m : M - 1) * x_stride;
    Piece<E> v[kQPieces];
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < kQPieces; ++c) {
      const int i = (c * lanes + lane) * N;
      if (i < K)
        v[c].load_upto(row + i, K - i);
      else
        v[c] = Piece<E>{};
    }
#pragma unroll
    for (int c = 0; c < kQPieces; ++c) top = top_bits(v[c], top);
    for (int i = (kQPieces * lanes + lane) * N; i < K; i += lanes * N) {
      Piece<E> u;
      u.load_upto(row + i, K - i);
      top = top_bits(u, top);
    }
    top = wave_umax32(as_f32_bits<E>(top));
    if (lanes > kWave) {
      __syncthreads();
      if ((threadIdx.x & 63) == 0) part[threadIdx.x / kWave] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kQThreads / kWave; ++w) top = max(top, part[w]);
    }
    const bool finite = top < 0x7F800000u;
    const float s = fmaxf(__uint_as_float(top) / 127.0f, kMinScale);
    const float inv = finite ? 1.0f / s : 0.0f;
    if (m >= M) continue;
    if (lane == 0) scale[m] = finite ? s : __uint_as_float(0x7FC00000u);
    int8_t* out = q + m * q_stride;
    auto put = [&](const Piece<E>& u, int i) {  // whole pieces: the row is padded to 16 bytes
      quantize_piece(finite ? u : Piece<E>{}, s, inv, out + i);
    };
#pragma unroll
    for (int c = 0; c < kQPieces; ++c) {
      const int i = (c * lanes + lane) * N;
      if (i < width) put(v[c], i);
    }
    for (int i = (kQPieces * lanes + lane) * N; i < width; i += lanes * N) {
      Piece<E> u{};
      if (i < K) u.load_upto(row + i, K - i);
      put(u, i);
    }
  }
}

// ---------------------------------------------------------------------------
// moe_int8_matmul
// ---------------------------------------------------------------------------
struct MatArgs {
  int M, N, K, G, a_rows, index_div, out_dtype;
  const int8_t* a;
  const float* a_scale;
  const int32_t* index;
  const int32_t* offsets;
  const int8_t* b;
  const float* b_scale;
  void* out;
  size_t a_stride, b_stride, b_group_stride, b_scale_group_stride, out_stride;
};

template <typename E>
__device__ __forceinline__ void store4(const MatArgs& p, int m, int n, const float (&y)[4]) {
  Piece<E, 4> o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.e[i] = from_f32<E>(y[i]);
  o.store_upto((E*)p.out + (size_t)m * p.out_stride + n, p.N - n);
}

__device__ __forceinline__ void store_out(const MatArgs& p, int m, int n, const float (&y)[4]) {
  if (p.out_dtype == MOE_DT_BF16)
    store4<Bf16>(p, m, n, y);
  else if (p.out_dtype == MOE_DT_FP16)
    store4<Fp16>(p, m, n, y);
  else
    store4<float>(p, m, n, y);
}

// 16 bytes at element k of a row, zero from element K on; 0 <= k < up16(K).
__device__ __forceinline__ i32x4 load_k(const int8_t* row, int k) {
  return *(const i32x4*)(row + k);
}
__device__ __forceinline__ i32x4 mask_k(i32x4 v, int valid) {  // the first `valid` bytes
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int left = valid - 4 * w;
    v[w] = left >= 4 ? v[w] : left <= 0 ? 0 : v[w] & (int)((1u << (8 * left)) - 1u);
  }
  return v;
}

// Streaming form, for products of few tiles: a workgroup takes 32 rows of b (with
// SwiGLU, 16 gate rows and their 16 up rows) and up to 16 * MT rows of one
// group, its W waves the chunks of 64 along K in turn; the integer sums are added
// through LDS.  b goes from memory straight to the registers of the matrix
// instruction (lane l: row l % 16, bytes 16 (l / 16) of the chunk), since nothing
// else in the workgroup uses it.  One row, K = 4096, 2N = 4096 (16.8 MB) takes 7.3
// us where the caches hold b and 8.7 from memory.  Bound by how much is in flight:
// the loads of kSUnroll chunks stand before their products, but the compiler moves
// them between, and the built kernel has those of two chunks (4 to 6 loads) under
// way and 71 registers; and one row of 2N = 4096 is 128 workgroups, half the CUs.
// Eight waves against four, one row: 7.5 us against 7.8; kSUnroll 8 against 4, four
// waves: 7.8 against 8.3; one row each of eight such groups: 33 us with eight waves
// against 29.8 with four.
constexpr int kSUnroll = 8;

template <int W, int MT, bool GLU>
__device__ __forceinline__ void stream_tile(const MatArgs& p, const Rows& r, int n0,
                                            i32x4 (&part)[W][MT * 2][kWave]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x / kWave;
  const int col = lane & 15, quad = lane >> 4;

  const int8_t* b = p.b + (size_t)r.g * p.b_group_stride;
  const int8_t* brow[2];
  brow[0] = b + (size_t)min(n0 + col, p.N - 1) * p.b_stride;
  brow[1] = b + (size_t)(GLU ? p.N + min(n0 + col, p.N - 1) : min(n0 + 16 + col, p.N - 1)) *
                    p.b_stride;
  const int8_t* arow[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int src = source_row(p, min(r.lo + 16 * t + col, r.hi - 1));
    arow[t] = p.a + (size_t)max(src, 0) * p.a_stride;
  }

  i32x4 acc[MT][2] = {};
  const int full = p.K / 64;  // chunks that lie inside the rows
  int c = wave;
  for (; c + W * (kSUnroll - 1) < full; c += W * kSUnroll) {
    i32x4 wb[kSUnroll][2], wa[kSUnroll][MT];
#pragma unroll
    for (int u = 0; u < kSUnroll; ++u) {
      const int k = 64 * (c + W * u) + 16 * quad;
#pragma unroll
      for (int s = 0; s < 2; ++s) wb[u][s] = load_k(brow[s], k);
#pragma unroll
      for (int t = 0; t < MT; ++t) wa[u][t] = load_k(arow[t], k);
    }
#pragma unroll
    for (int u = 0; u < kSUnroll; ++u)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int s = 0; s < 2; ++s)
          acc[t][s] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wb[u][s], wa[u][t], acc[t][s], 0, 0, 0);
  }
  for (; 64 * c < p.K; c += W) {
    const int k = 64 * c + 16 * quad, valid = p.K - k;
    const int at = valid > 0 ? k : 0;  // a piece past the row is read from its start and zeroed
    i32x4 wb[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) wb[s] = load_k(brow[s], at);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const i32x4 wa = mask_k(load_k(arow[t], at), valid);
#pragma unroll
      for (int s = 0; s < 2; ++s)
        acc[t][s] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wb[s], wa, acc[t][s], 0, 0, 0);
    }
  }

#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int s = 0; s < 2; ++s) part[wave][t * 2 + s][lane] = acc[t][s];
  __syncthreads();
  for (int t = wave; t < MT; t += W) {
    i32x4 sum[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      sum[s] = part[0][t * 2 + s][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) sum[s] += part[w][t * 2 + s][lane];
    }
    // lane: row `col` of out, columns 4 * quad .. + 3 of each 16
    const int m = r.lo + 16 * t + col;
    if (m >= r.hi) continue;
    const int src = source_row(p, m);
    if (src < 0) continue;
    const float sa = p.a_scale[src];
    const float* sb = p.b_scale + (size_t)r.g * p.b_scale_group_stride;
    float y[2][4];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + 4 * quad + i + (GLU ? 0 : 16 * s);
        const float sn = sb[min(n, p.N - 1) + (GLU && s ? p.N : 0)];
        y[s][i] = (float)sum[s][i] * sa * sn;
      }
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

template <int W, int MT, bool GLU>
__global__ __launch_bounds__(W* kWave) void int8_stream(MatArgs p, int cols, int64_t first) {
  __shared__ i32x4 part[W][MT * 2][kWave];
  __shared__ int counts[W];
  const int64_t w = first + blockIdx.x;
  Rows r;
  if (!find_rows(p, w / cols, 16 * MT, counts, r)) return;
  stream_tile<W, MT, GLU>(p, r, (int)(w % cols) * (GLU ? 16 : 32), part);
}

template <int W, int MT>
void launch_stream_of(const MatArgs& p, bool glu, int cols, int64_t tiles, hipStream_t stream) {
  for (int64_t first = 0; first < tiles; first += kMaxGrid) {
    const unsigned grid = (unsigned)(tiles - first < kMaxGrid ? tiles - first : kMaxGrid);
    if (glu)
      int8_stream<W, MT, true><<<grid, W * kWave, 0, stream>>>(p, cols, first);
    else
      int8_stream<W, MT, false><<<grid, W * kWave, 0, stream>>>(p, cols, first);
  }
}

template <int MT>
void launch_stream(const MatArgs& p, bool glu, hipStream_t stream) {
  const int per = glu ? 16 : 32, cols = (p.N + per - 1) / per;
  const int64_t tiles = max_items(p.M, p.G, 16 * MT) * cols;
  if (tiles <= 512)  // two for each CU: more waves, so that enough is in flight
    launch_stream_of<8, MT>(p, glu, cols, tiles, stream);
  else
    launch_stream_of<4, MT>(p, glu, cols, tiles, stream);
}

// Tiled form, for groups of more rows: a workgroup of eight waves, two by four,
// takes 32 * MF rows of one group and 256 rows of b (with SwiGLU, 128 gate rows
// and their 128 up rows); a wave has 16 * MF rows by 64.  Both operands go
// through LDS by direct loads, in a ring of S stages of 128 bytes of K: whole
// cache lines of a row, which the memory path takes fastest.  (b straight to
// the registers of the waves that use it, 16 rows x 64 bytes a load, left the
// loads alone at 496 us of dense 8192^3, where the tile as it is takes 413.)
//
// A tile of 256 x 256 loads 64 KB a stage for 33.6 M products, so with a few
// hundred rows in each group it is the matrix cores that bound: they are busy 56 %
// of the cycles of the long gate/up products, at the 1.6 to 1.7 GHz that they are
// held to under that load; LDS conflicts are 1 % of its accesses.  Dense 8192^3
// takes 402 to 413 us (2.67 to 2.73 POPS), 65536 rows over 130 groups (K 6144, 2N
// 4096) 1.59 to 1.62 ms (2.07 POPS of exact work, tiles' empty rows not counted;
// 1.54 to 1.76 ms call by call under a trace).  With few rows in each group the
// weights bound: 5.3 to 5.7 TB/s at one decode step, 5.2 at 16384 rows over 166.
constexpr int kTWaves = 8;
constexpr int kStep = 128;  // bytes of K a stage
constexpr int kColRows = 256;

// What the epilogue needs of a tile's rows and columns, loaded beside the first
// stage.
constexpr int kMostRows = 320;

struct Side {
  float row[kMostRows], col[kColRows];
  int live[kMostRows];  // rows of out that are written
};

constexpr int kOutBytes = 16384;  // LDS that a wave's results pass through

// ONCE: these are all rows of their group, so b is read by this workgroup alone
// and passes the caches by (one decode step's gate/up, 761 MB: 147 us against
// 134; 16384 rows over 166 groups, down: 310 against 305).
template <typename E, int MF, int S, bool GLU, bool ONCE>
__device__ __forceinline__ void tile(const MatArgs& p, const Rows& r, int n0, uint8_t* smem,
                                     Side& side) {
  constexpr int kRows = 32 * MF;
  constexpr int kStage = (kRows + kColRows) * kStep;  // bytes of a stage, rows of a first
  constexpr int kLoadsA = kRows / 8 / kTWaves;        // direct loads of a wave, 8 rows each
  constexpr int kLoadsB = kColRows / 8 / kTWaves;
  constexpr int kLoads = kLoadsA + kLoadsB;
  constexpr int kOut = GLU ? 8 : 16;                  // consecutive columns a lane ends with
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int col = lane & 15, quad = lane >> 4;
  const int wm = wave >> 2, wn = wave & 3;

  // Direct loads: a lane loads 16 bytes of row lane / 8 of its instruction's
  // eight.  LDS place (row, c) holds piece c ^ (row & 7) of the row's 128 bytes,
  // so that the 16 rows of a fragment spread over the banks.
  const int piece = 16 * ((lane & 7) ^ (lane >> 3));
  // LDS row 64 w + 16 s + x of b is row x of fragment s of the waves wn = w: the
  // weight row that gives lane quad q of the result the columns kOut * q + 4 * s
  // + i, so that a lane ends with kOut consecutive columns of out.
  const int8_t* brow[kLoadsB];
#pragma unroll
  for (int j = 0; j < kLoadsB; ++j) {
    const int l = (wave * kLoadsB + j) * 8 + (lane >> 3);
    const int s = (l >> 4) & 3, x = l & 15;
    const int n = n0 + (l >> 6) * 4 * kOut + kOut * (x >> 2) + 4 * (GLU ? s & 1 : s) + (x & 3);
    brow[j] = p.b + (size_t)r.g * p.b_group_stride +
              (size_t)(min(n, p.N - 1) + (GLU && s >= 2 ? p.N : 0)) * p.b_stride + piece;
  }
  const int steps = (p.K + kStep - 1) / kStep;
  const int width = up16(p.K);

  // Loads of stage i.  Behind a row, b's pieces are zero, and a's any bytes of
  // the row.
  auto load_b = [&](int i, int j) {
    const int k = i * kStep;
    const uint8_t* from = k + piece < width ? (const uint8_t*)brow[j] + k : kZeros;
    uint8_t* to = smem + (i % S) * kStage + kRows * kStep + (wave * kLoadsB + j) * 1024;
    if (ONCE)
      dma16_past(from, to);
    else
      dma16(from, to);
  };
#pragma unroll
  for (int j = 0; j < kLoadsB; ++j) load_b(0, j);
  const int8_t* arow[kLoadsA];
#pragma unroll
  for (int j = 0; j < kLoadsA; ++j) {
    const int m = r.lo + (wave * kLoadsA + j) * 8 + (lane >> 3);
    arow[j] = p.a + (size_t)max(source_row(p, min(m, r.hi - 1)), 0) * p.a_stride + piece;
  }
  auto load_a = [&](int i, int j) {
    const int k = i * kStep;
    dma16((const uint8_t*)arow[j] + (k + piece < width ? k : -piece),
          smem + (i % S) * kStage + (wave * kLoadsA + j) * 1024);
  };
  auto load = [&](int i, int j) {
    if (j < kLoadsB)
      load_b(i, j);
    else
      load_a(i, j - kLoadsB);
  };

  // One stage: 2 * MF groups of four products, a group for each 64 bytes of 16
  // rows of a.  Fragments are read two groups ahead (b's a half stage ahead), and
  // the loads of stage i + S - 1 are issued one for each group.  A wave at its
  // products goes before the SIMD's other one at its loads (dense 8192^3 449 us
  // against 427).
  i32x4 acc[MF][4] = {};
  auto stage = [&](int i, auto more) {
    const uint8_t* sa = smem + (i % S) * kStage + (wm * MF * 16 + col) * kStep;
    const uint8_t* sb = smem + (i % S) * kStage + (kRows + wn * 64 + col) * kStep;
    const int slot[2] = {16 * (quad ^ (col & 7)), 16 * ((4 + quad) ^ (col & 7))};
    auto frag = [&](int x) { return *(const i32x4*)(sa + (x % MF) * 16 * kStep + slot[x / MF]); };
    auto weight = [&](int c, int s) { return *(const i32x4*)(sb + s * 16 * kStep + slot[c]); };
    i32x4 w[3], v[2][4];
#pragma unroll
    for (int s = 0; s < 4; ++s) v[0][s] = weight(0, s);
    w[0] = frag(0);
    w[1] = frag(1);
#pragma unroll
    for (int x = 0; x < 2 * MF; ++x) {
      if (x + 2 < 2 * MF) w[(x + 2) % 3] = frag(x + 2);
#pragma unroll
      for (int s = x; x < MF && s < 4; s += MF) v[1][s] = weight(1, s);
      if (decltype(more)::value) {
#pragma unroll
        for (int j = x; j < kLoads; j += 2 * MF) load(i + S - 1, j);
      }
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int s = 0; s < 4; ++s)
        acc[x % MF][s] = __builtin_amdgcn_mfma_i32_16x16x64_i8(v[x / MF][s], w[x % 3],
                                                               acc[x % MF][s], 0, 0, 0);
      __builtin_amdgcn_s_setprio(0);
    }
  };

#pragma unroll
  for (int i = 0; i < S - 1; ++i)
    if (i < steps)
      for (int j = i ? 0 : kLoadsB; j < kLoads; ++j) load(i, j);
  for (int t = threadIdx.x; t < kRows; t += kTWaves * kWave) {
    const int src = r.lo + t < r.hi ? source_row(p, r.lo + t) : -1;
    side.live[t] = src >= 0;
    side.row[t] = src >= 0 ? p.a_scale[src] : 0.0f;
  }
  for (int t = threadIdx.x; t < kColRows; t += kTWaves * kWave) {
    const int n = n0 + (GLU ? t & 127 : t);
    side.col[t] = p.b_scale[(size_t)r.g * p.b_scale_group_stride + min(n, p.N - 1) +
                            (GLU && t >= 128 ? p.N : 0)];
  }
  // At the top of stage i its loads, issued S - 1 stages ago, have to have
  // landed (those of the S - 2 stages after it may still be in flight), and
  // every wave has to be done with the stage before, whose place is loaded next.
  int i = 0;
  for (; i + S - 1 < steps; ++i) {
    wait_loads<(S - 2) * kLoads>();
    barrier();
    stage(i, std::true_type{});
  }
  wait_loads<0>();
  barrier();
  if (p.K % 16 != 0) {  // the end of the row cuts a piece of the last stage: zeros from there on
    const int k = p.K / 16 * 16 - (steps - 1) * kStep;
    for (int x = threadIdx.x; x < kColRows; x += kTWaves * kWave) {
      i32x4* at = (i32x4*)(smem + ((steps - 1) % S) * kStage + (kRows + x) * kStep +
                           (k ^ (16 * (x & 7))));
      *at = mask_k(*at, p.K % 16);
    }
    barrier();
  }
  for (; i < steps; ++i) stage(i, std::false_type{});

  // Results leave through LDS, each wave through a part of its own, so that
  // eight lanes store 128 consecutive bytes of a row of out.  16 bytes c of row
  // x lie at c ^ (x & 7) of each 128, for the banks.  The stores pass the caches
  // by, which leaves these to a and b (8192 x 8192 x 2048 137 us against 121).
  constexpr int kRowBytes = 4 * kOut * (int)sizeof(E);    // a wave's part of a row of out
  constexpr int kPartRows = kOutBytes / kRowBytes;        // rows that pass at a time
  constexpr int kPart = part_of(MF, kPartRows / 16);      // fragments of them
  constexpr int kPieces = kRowBytes / 16;
  float sn[4][4];
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      sn[s][e] = side.col[(GLU && s >= 2 ? 128 : 0) + (wn * 4 + quad) * kOut +
                          4 * (GLU ? s & 1 : s) + e];
  barrier();  // every wave has read the last stage
  uint8_t* mine = smem + wave * kOutBytes;
  auto place = [&](int x, int c) { return mine + x * kRowBytes + 16 * (c ^ (x & (kPieces - 1) & 7)); };
#pragma unroll
  for (int f0 = 0; f0 < MF; f0 += kPart) {
#pragma unroll
    for (int f = f0; f < f0 + kPart; ++f) {
      const float sa = side.row[(wm * MF + f) * 16 + col];
      Piece<E, kOut> o;
      float y[kOut];
#pragma unroll
      for (int j = 0; j < kOut; ++j) y[j] = (float)acc[f][j / 4][j % 4] * sa * sn[j / 4][j % 4];
      if constexpr (GLU) {
        float up[kOut], h[kOut];
#pragma unroll
        for (int j = 0; j < kOut; ++j)
          up[j] = (float)acc[f][2 + j / 4][j % 4] * sa * sn[2 + j / 4][j % 4];
        swiglu(y, up, h);
#pragma unroll
        for (int j = 0; j < kOut; ++j) o.e[j] = from_f32<E>(h[j]);
      } else {
#pragma unroll
        for (int j = 0; j < kOut; ++j) o.e[j] = from_f32<E>(y[j]);
      }
      constexpr int kMine = kOut * (int)sizeof(E) / 16;
#pragma unroll
      for (int c = 0; c < kMine; ++c)
        __builtin_memcpy(place((f - f0) * 16 + col, quad * kMine + c), (const char*)o.e + 16 * c, 16);
    }
    wave_exchange();
    constexpr int kPer = 64 / kPieces;  // rows of a store instruction
#pragma unroll
    for (int x0 = 0; x0 < kPart * 16; x0 += kPer) {
      const int x = x0 + lane / kPieces, c = lane % kPieces;
      Piece<E> o;
      __builtin_memcpy(o.e, place(x, c), 16);
      const int row = (wm * MF + f0) * 16 + x, n = n0 + wn * 4 * kOut + c * Piece<E>::kN;
      if (!side.live[row] || n >= p.N) continue;
      E* to = (E*)p.out + (size_t)(r.lo + row) * p.out_stride + n;
      if (p.N - n >= Piece<E>::kN)
        o.store_past(to);
      else
        o.store_head(to, p.N - n);
    }
    wave_exchange();  // the part is written over next
  }
}

template <typename E, bool GLU>
__global__ __launch_bounds__(kTWaves* kWave, 2) void int8_tiles(MatArgs p, int R, int cols,
                                                               bool blocks, int64_t first) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * (kMostRows + kColRows) * kStep];
  __shared__ Side side;
  __shared__ int counts[kTWaves];
  int64_t item;
  int col;
  Rows r;
  tile_of(first + blockIdx.x, blocks, cols, item, col);
  if (col >= cols || !find_rows(p, item, R, counts, r)) return;
  const int n0 = col * (GLU ? kColRows / 2 : kColRows), rows = r.hi - r.lo;
  if (rows <= 64 && r.all)
    tile<E, 2, 3, GLU, true>(p, r, n0, smem, side);
  else if (rows <= 64)
    tile<E, 2, 3, GLU, false>(p, r, n0, smem, side);
  else if (rows <= 128 && r.all)
    tile<E, 4, 3, GLU, true>(p, r, n0, smem, side);
  else if (rows <= 128)
    tile<E, 4, 3, GLU, false>(p, r, n0, smem, side);
  else if (rows <= 192)
    tile<E, 6, 2, GLU, false>(p, r, n0, smem, side);
  else if (rows <= 256)
    tile<E, 8, 2, GLU, false>(p, r, n0, smem, side);
  else
    tile<E, 10, 2, GLU, false>(p, r, n0, smem, side);
}

// Most rows of a tile.  More rows share a load of b's, but a product of few tiles
// may then leave more of the 256 CUs without one: its time goes as rounds *
// (rows + 256), the bytes that a tile loads in a stage (512 x 4096 x 4096: 48 us
// with 320 rows, 21 with 64).  Groups that fill the CUs get the most rows, so
// that more of them read their weights once.
int rows_of_tile(const MatArgs& p, int cols) {
  const int64_t groups = p.G > 0 ? (p.G < p.M ? p.G : p.M) : 0;
  if (groups > 0 && (p.M / kMostRows + groups) * cols >= 256) return kMostRows;
  int best = kMostRows;
  int64_t least = INT64_MAX;
  for (int R : {320, 256, 192, 128, 64}) {
    const int64_t items = groups > 0 ? p.M / R + groups : ((int64_t)p.M + R - 1) / R;
    const int64_t cost = (items * cols + 255) / 256 * (R + 256);
    if (cost < least) best = R, least = cost;
  }
  return best;
}

// The streaming form is for products whose tiles, of 64 rows even, would leave
// most CUs idle: at N = K = 4096, dense, 128 rows take 17 us against 20 in tiles
// and 160 rows 24 against 20.  Groups of few rows are bound by their weights,
// which more workgroups read faster: with 4096 gate and up rows, 8 groups of one
// row take 30 us against 34 and 16 groups 54 against 51.
bool few_tiles(const MatArgs& p, bool glu) {
  const int64_t cols = ((int64_t)p.N + (glu ? 127 : 255)) / (glu ? 128 : 256);
  int64_t items = ((int64_t)p.M + 63) / 64;
  bool thin = false;
  if (p.G > 0) {
    const int64_t groups = p.G < p.M ? p.G : p.M;
    if (items < groups) items = groups;
    thin = p.M < 4 * groups;
  }
  return items * cols < (thin ? 192 : 48);
}

template <typename E>
void launch_tiles(const MatArgs& p, bool glu, hipStream_t stream) {
  const int per = glu ? kColRows / 2 : kColRows, cols = (p.N + per - 1) / per;
  const int R = rows_of_tile(p, cols);
  const int64_t items = max_items(p.M, p.G, R);
  // Blocks pay where b is read by several tiles (65536 rows over 130 groups, gate/up
  // 1642 us against 1605, down 910 against 891) and each XCD has many of them;
  // weights that are read once gain nothing (16384 rows over 166 groups: 303).
  const bool blocks = p.M > 128 * (int64_t)(p.G > 0 ? p.G : 1) && items * cols >= 2048;
  const int64_t tiles =
      blocks ? (int64_t)up_to((items + kBlockItems - 1) / kBlockItems *
                                  ((cols + kBlockCols - 1) / kBlockCols), 8) *
                   kBlockItems * kBlockCols
             : items * cols;
  for (int64_t first = 0; first < tiles; first += kMaxGrid) {
    const unsigned grid = (unsigned)(tiles - first < kMaxGrid ? tiles - first : kMaxGrid);
    if (glu)
      int8_tiles<E, true><<<grid, kTWaves * kWave, 0, stream>>>(p, R, cols, blocks, first);
    else
      int8_tiles<E, false><<<grid, kTWaves * kWave, 0, stream>>>(p, R, cols, blocks, first);
  }
}

int matmul_status(const moe_int8_matmul_args* a) {
  if (!a) return MOE_EINVAL;
  if (a->M < 0 || a->N <= 0 || a->K <= 0 || a->G < 0 || a->a_rows < 0) return MOE_EINVAL;
  if (dtype_bytes(a->out_dtype) == 0 || (a->swiglu != 0 && a->swiglu != 1)) return MOE_EINVAL;
  if (a->K > kMaxK || a->G > MOE_MAX_S || a->N > (1 << 24) || a->M > (1 << 30))
    return MOE_EUNSUPPORTED;
  if (a->M == 0) return MOE_OK;
  if (!a->a || !a->a_scale || !a->b || !a->b_scale || !a->out) return MOE_EINVAL;
  if ((a->G > 0) != (a->offsets != nullptr)) return MOE_EINVAL;
  if (a->index ? a->index_div < 1 : a->a_rows < a->M) return MOE_EINVAL;
  if (a->a_rows == 0) return MOE_EINVAL;
  const size_t row = (size_t)up16(a->K), wide = (size_t)a->N * (a->swiglu ? 2 : 1);
  if (!aligned(a->a, 16) || !aligned(a->b, 16) || a->a_stride % 16 || a->b_stride % 16 ||
      a->b_group_stride % 16)
    return MOE_EINVAL;
  if (!aligned(a->a_scale, 4) || !aligned(a->b_scale, 4) || !aligned(a->index, 4) ||
      !aligned(a->offsets, 4) || !aligned(a->out, dtype_bytes(a->out_dtype)))
    return MOE_EINVAL;
  if (a->a_stride < row || a->b_stride < row || a->out_stride < (size_t)a->N) return MOE_EINVAL;
  if (a->G > 1 && (a->b_group_stride < (wide - 1) * a->b_stride + row ||
                   a->b_scale_group_stride < wide))
    return MOE_EINVAL;
  return MOE_OK;
}

}  // namespace

extern "C" MOE_EXPORT size_t moe_int8_row_bytes(int K) {
  return K <= 0 || K > kMaxK ? 0 : (size_t)up16(K);
}

extern "C" MOE_EXPORT int moe_int8_quantize(const void* x, int M, int K, size_t x_stride, int dtype,
                                            int8_t* q, size_t q_stride, float* scale,
                                            hipStream_t stream) {
  const size_t e = dtype_bytes(dtype);
  if (M < 0 || K <= 0 || e == 0) return MOE_EINVAL;
  if (K > kMaxK) return MOE_EUNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!x || !q || !scale || !aligned(x, e) || !aligned(q, 16) || !aligned(scale, 4))
    return MOE_EINVAL;
  if (x_stride < (size_t)K || q_stride % 16 || q_stride < (size_t)up16(K)) return MOE_EINVAL;
  const int pieces = (K * (int)e + 15) / 16;
  const int lanes = pieces <= kWave * kQPieces ? kWave : kQThreads;
  const int64_t want = ((int64_t)M * lanes + kQThreads - 1) / kQThreads;
  const unsigned grid = (unsigned)(want < kMaxGrid ? want : kMaxGrid);
  if (dtype == MOE_DT_BF16)
    quantize_rows<Bf16><<<grid, kQThreads, 0, stream>>>((const Bf16*)x, M, K, x_stride, q, q_stride,
                                                        scale, lanes);
  else if (dtype == MOE_DT_FP16)
    quantize_rows<Fp16><<<grid, kQThreads, 0, stream>>>((const Fp16*)x, M, K, x_stride, q, q_stride,
                                                        scale, lanes);
  else
    quantize_rows<float><<<grid, kQThreads, 0, stream>>>((const float*)x, M, K, x_stride, q,
                                                         q_stride, scale, lanes);
  return hip_status();
}

extern "C" MOE_EXPORT int moe_int8_matmul(const moe_int8_matmul_args* a, hipStream_t stream) {
  const int s = matmul_status(a);
  if (s != MOE_OK || a->M == 0) return s;
  MatArgs p{};
  p.M = a->M, p.N = a->N, p.K = a->K, p.G = a->G;
  p.a_rows = a->a_rows, p.index_div = a->index_div, p.out_dtype = a->out_dtype;
  p.a = a->a, p.a_scale = a->a_scale, p.index = a->index, p.offsets = a->offsets;
  p.b = a->b, p.b_scale = a->b_scale, p.out = a->out;
  p.a_stride = a->a_stride, p.b_stride = a->b_stride, p.b_group_stride = a->b_group_stride;
  p.b_scale_group_stride = a->b_scale_group_stride, p.out_stride = a->out_stride;
  if (few_tiles(p, a->swiglu)) {
    const int rows = p.M / (p.G > 0 ? (p.G < p.M ? p.G : p.M) : 1);  // of a group, on average
    if (rows <= 32)
      launch_stream<1>(p, a->swiglu, stream);
    else if (rows <= 64)
      launch_stream<2>(p, a->swiglu, stream);
    else
      launch_stream<4>(p, a->swiglu, stream);
  } else if (p.out_dtype == MOE_DT_BF16) {
    launch_tiles<Bf16>(p, a->swiglu, stream);
  } else if (p.out_dtype == MOE_DT_FP16) {
    launch_tiles<Fp16>(p, a->swiglu, stream);
  } else {
    launch_tiles<float>(p, a->swiglu, stream);
  }
  return hip_status();
}
