// Tiled products of ragged groups of rows in floating point: the kernels that
// grouped_bf16.hip, grouped_fp16.hip and grouped_fp32.hip build for their type.
//
//   rows   out[p,n] = sum_k a[r(p),k] * b[g,n,k]     rows p of group g
//   outer  out[g,l,r] = sum_p left[p,l] * right[p,r]
//
// Both are tiles of a left operand against a right one over a contraction.  An
// operand lies with its contraction along the rows of memory (a, and b of layout
// [N][K]) or across them (b of layout [K][N], left and right of outer).  It is
// staged in LDS as it lies, in whole pieces of 16 bytes; one that lies across is
// read from LDS by the transposing loads, four contraction steps a lane.
#pragma once

#include <type_traits>

#include "groups.hpp"

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct RowsProduct {
  int M, N, K, G, a_rows, index_div;  // N: columns of out; with SwiGLU b has 2N
  const void *a, *b;
  void* out;
  float* pre;  // the products before SwiGLU, [M][2N], or null
  const int32_t *index, *offsets;
  const int32_t* pos;  // the row of each of M assignments, or null: the only one that index names
  size_t a_stride, b_stride, b_group_stride, out_stride, pre_stride;  // elements
  bool zero_rest;  // rows that nothing is computed for become zero
  bool out_f32;    // out is float32 whatever the element type
};

struct OuterProduct {
  int M, L, R, G, left_rows, right_rows, left_div, right_div;
  const void *left, *right;
  void* out;
  const int32_t *left_index, *right_index, *offsets;
  const int32_t* pos;  // as in RowsProduct, for the operand that has an index
  size_t left_stride, right_stride, out_stride, out_group_stride;  // elements
  int splits;   // parts of each group's rows, with sums of their own
  float* sums;  // [splits][G][L][R], or null for one part
};

template <typename E>
int launch_rows_product(const RowsProduct& p, bool across, bool glu, hipStream_t stream);
template <typename E>
int launch_outer_product(const OuterProduct& p, hipStream_t stream);

// The assignment that row m has of `index`; -1 for none, or with pos for one whose row is
// another.
__device__ __forceinline__ int named_at(const int32_t* index, const int32_t* pos, int M, int m) {
  const int r = index[m];
  if (!pos || (unsigned)r >= (unsigned)M) return r < 0 ? -1 : r;
  return pos[r] == m ? r : -1;
}
__device__ __forceinline__ int source_row(const RowsProduct& p, int m) {
  int r = m;
  if (p.index) {
    r = named_at(p.index, p.pos, p.M, m);
    r = r < 0 ? -1 : r / p.index_div;
  }
  return (unsigned)r < (unsigned)p.a_rows ? r : -1;
}

// acc += products of 16 x 16 fragments over 64 bytes of contraction, sums in float32.
// A lane holds 16 bytes of row (lane & 15) from byte 16 * (lane >> 4) on; it gets rows
// 4 * (lane >> 4) .. + 3 of w against row (lane & 15) of x.
template <typename E>
__device__ __forceinline__ f32x4 mma(i32x4 w, i32x4 x, f32x4 acc);
template <>
__device__ __forceinline__ f32x4 mma<Bf16>(i32x4 w, i32x4 x, f32x4 acc) {
  typedef __bf16 V __attribute__((ext_vector_type(8)));
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(V, w),
                                                 __builtin_bit_cast(V, x), acc, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mma<Fp16>(i32x4 w, i32x4 x, f32x4 acc) {
  typedef _Float16 V __attribute__((ext_vector_type(8)));
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(V, w),
                                                __builtin_bit_cast(V, x), acc, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mma<float>(i32x4 w, i32x4 x, f32x4 acc) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__int_as_float(w[e]), __int_as_float(x[e]), acc, 0,
                                               0, 0);
  return acc;
}

constexpr int kStep = 128;     // bytes of contraction a stage
constexpr int kMostRows = 320;

// A workgroup has two waves down by WA across; a wave has 64 columns.
template <int WA>
struct Wide {
  static constexpr int kCols = 64 * WA, kWaves = 2 * WA, kThreads = kWaves * kWave;
};
constexpr int kSmall = 1, kLarge = 4;  // WA of products of few tiles, and of the others
template <typename E>
constexpr int kOuter = sizeof(E) == 4 ? 2 : 4;  // of outer products: tiles of 64 kOuter squared

// Where an operand that lies across its contraction is in LDS: a stage is kStep /
// sizeof(E) rows of W elements, 16-byte pieces of a row swapped so that the places
// one read takes in 16 rows spread over the banks.
template <typename E, int W>
__device__ __forceinline__ int swap_piece(int piece, int row) {
  if constexpr (sizeof(E) == 2) {
    constexpr int kUnits = W / 16;  // 32 bytes, the 16 columns of a fragment
    const int g = ((row & 3) | ((row >> 3) & 3) << 2) & (kUnits - 1);
    return piece ^ (2 * g);
  } else {
    return piece ^ (4 * ((row >> 2) & 3));
  }
}

// 16 bytes of contraction of the lane's column (lane & 15) from column `at` on, half
// `half` of the stage.
template <typename E, int W>
__device__ __forceinline__ i32x4 read_across(const uint8_t* stage, int at, int half) {
  const int lane = threadIdx.x & 63, x = lane & 15, quad = lane >> 4;
  constexpr int kRow = W * (int)sizeof(E);
  i32x4 v;
  if constexpr (sizeof(E) == 2) {
    typedef short V __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) V LV;
    typedef int I2 __attribute__((ext_vector_type(2)));
    const int row = 32 * half + 8 * quad + (x >> 2);
    const int c = at / 8 + ((x & 3) >> 1);
    const uint8_t* from =
        stage + row * kRow + 16 * swap_piece<E, W>(c, row) + 8 * (x & 1);
    const I2 lo = __builtin_bit_cast(I2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LV*)from));
    const I2 hi =
        __builtin_bit_cast(I2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LV*)(from + 4 * kRow)));
    v[0] = lo[0], v[1] = lo[1], v[2] = hi[0], v[3] = hi[1];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = 16 * half + 4 * quad + e;
      v[e] = *(const int*)(stage + row * kRow + 16 * swap_piece<E, W>((at + x) / 4, row) +
                           4 * (x & 3));
    }
  }
  return v;
}

// What a load of a stage takes: 16 bytes at p, of which n elements count (n <= 0: none).
template <typename E>
struct Src {
  const E* p;
  int n;
};

// The main loop.  A stage holds 32 * MF rows (LEFT across: columns) of the left
// operand and 64 * WA of the right one, kStep bytes of contraction each, in a ring of S; from_left(i, j,
// row, piece) and from_right say where the 16-byte piece of stage i is in memory that the
// wave's load j of the operand takes, `row` the row (across: the contraction step) and
// `piece` the piece in it; before(i) is called ahead of the loads of stage i.  DMA: loads go to
// LDS directly, and pieces count whole or not at all; otherwise they pass through
// registers, from any address and cut at any element.
//
// A wave has 16 * MF rows by 64 columns.  Its fragments are read two groups of products
// ahead (the right operand's a half stage ahead), and the loads of stage i + S - 1 are
// issued one for each group; a wave at its products goes before the SIMD's other one at
// its loads.
template <typename E, bool LEFT, bool RIGHT, bool SPLIT, int WA, int MF, int S, bool DMA,
          bool ONCE, typename FB, typename FL, typename FR>
__device__ __forceinline__ void products(uint8_t* smem, int steps, FB before, FL from_left,
                                         FR from_right, f32x4 (&acc)[MF][4]) {
  constexpr int kRows = 32 * MF, kCols = Wide<WA>::kCols, kWaves = Wide<WA>::kWaves;
  constexpr int kStage = (kRows + kCols) * kStep;
  constexpr int kLoadsL = kRows / 8 / kWaves, kLoadsR = kCols / 8 / kWaves;
  static_assert(kLoadsL * 8 * kWaves == kRows, "whole loads");
  constexpr int kLoads = kLoadsL + kLoadsR;
  constexpr int kPiece = 16 / (int)sizeof(E);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int col = lane & 15, quad = lane >> 4;
  const int wm = wave / WA, wn = wave % WA;

  // load j of a wave: LDS bytes 1024 * (wave * n + j) + 16 * lane of the operand's part
  auto source = [&](int i, int j) {
    if (j < kLoadsR) {
      const int u = (wave * kLoadsR + j) * 64 + lane;
      if constexpr (RIGHT) {
        const int row = u / (kCols / kPiece);
        return from_right(i, j, row, swap_piece<E, kCols>(u % (kCols / kPiece), row));
      } else {
        return from_right(i, j, u / 8, (u & 7) ^ ((u >> 3) & 7));
      }
    }
    const int u = (wave * kLoadsL + j - kLoadsR) * 64 + lane;
    if constexpr (LEFT) {
      const int row = u / (kRows / kPiece);
      return from_left(i, j - kLoadsR, row, swap_piece<E, kRows>(u % (kRows / kPiece), row));
    } else {
      return from_left(i, j - kLoadsR, u / 8, (u & 7) ^ ((u >> 3) & 7));
    }
  };
  auto place = [&](int i, int j) {  // of the wave's load j
    return smem + (i % S) * kStage +
           (j < kLoadsR ? kRows * kStep + (wave * kLoadsR + j) * 1024
                        : (wave * kLoadsL + j - kLoadsR) * 1024);
  };
  auto load = [&](int i, int j) {
    const Src<E> s = source(i, j);
    const uint8_t* from = s.n > 0 ? (const uint8_t*)s.p : kZeros;
    if (ONCE && j < kLoadsR)
      dma16_past(from, place(i, j));
    else
      dma16(from, place(i, j));
  };

  // float32 products are summed stage by stage: a chain of K / 32 and eight additions in
  // place of K / 4 (K 2900: relative error 1.2e-6 of an output against 5e-7)
  constexpr bool kApart = sizeof(E) == 4;
  f32x4 total[kApart ? MF : 1][4];
  if constexpr (kApart) {
#pragma unroll
    for (int f = 0; f < MF; ++f)
#pragma unroll
      for (int s = 0; s < 4; ++s) total[f][s] = acc[f][s], acc[f][s] = f32x4{};
  }
  auto stage = [&](int i, auto more) {
    const uint8_t* at = smem + (i % S) * kStage;
    const int slot[2] = {16 * (quad ^ (col & 7)), 16 * ((4 + quad) ^ (col & 7))};
    auto frag = [&](int x) -> i32x4 {
      if constexpr (LEFT)
        return read_across<E, kRows>(at, (wm * MF + x % MF) * 16, x / MF);
      else
        return *(const i32x4*)(at + ((wm * MF + x % MF) * 16 + col) * kStep + slot[x / MF]);
    };
    auto weight = [&](int c, int s) -> i32x4 {
      const uint8_t* r = at + kRows * kStep;
      if constexpr (RIGHT)
        return read_across<E, kCols>(
            r, SPLIT ? (s >= 2 ? kCols / 2 : 0) + wn * 32 + 16 * (s & 1) : wn * 64 + 16 * s, c);
      else
        return *(const i32x4*)(r + (wn * 64 + 16 * s + col) * kStep + slot[c]);
    };
    i32x4 w[3], v[2][4];
    if constexpr (decltype(more)::value) before(i + S - 1);
#pragma unroll
    for (int s = 0; s < 4; ++s) v[0][s] = weight(0, s);
    w[0] = frag(0);
    w[1] = frag(1);
#pragma unroll
    for (int x = 0; x < 2 * MF; ++x) {
      if (x + 2 < 2 * MF) w[(x + 2) % 3] = frag(x + 2);
#pragma unroll
      for (int s = x; x < MF && s < 4; s += MF) v[1][s] = weight(1, s);
      if constexpr (decltype(more)::value) {
#pragma unroll
        for (int j = x; j < kLoads; j += 2 * MF) load(i + S - 1, j);
      }
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int s = 0; s < 4; ++s) acc[x % MF][s] = mma<E>(v[x / MF][s], w[x % 3], acc[x % MF][s]);
      __builtin_amdgcn_s_setprio(0);
    }
    if constexpr (kApart) {
#pragma unroll
      for (int f = 0; f < MF; ++f)
#pragma unroll
        for (int s = 0; s < 4; ++s) total[f][s] += acc[f][s], acc[f][s] = f32x4{};
    }
  };

  if constexpr (DMA) {
    // At the top of stage i its loads, issued S - 1 stages ago, have to have landed
    // (those of the S - 2 stages after it may still be in flight), and every wave has to
    // be done with the stage before, whose place is loaded next.
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
      if (i < steps) {
        before(i);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) load(i, j);
      }
    int i = 0;
    for (; i + S - 1 < steps; ++i) {
      wait_loads<(S - 2) * kLoads>();
      barrier();
      stage(i, std::true_type{});
    }
    wait_loads<0>();
    barrier();
    for (; i < steps; ++i) stage(i, std::false_type{});
  } else {
    Piece<E> u[kLoads];
    auto fetch = [&](int i) {
      before(i);
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const Src<E> s = source(i, j);
        if (s.n > 0)
          u[j].load_upto(s.p, s.n);
        else
          u[j] = Piece<E>{};
      }
    };
    auto put = [&](int i) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) __builtin_memcpy(place(i, j) + 16 * lane, u[j].e, 16);
    };
    static_assert(S == 2, "two stages");
    if (steps > 0) fetch(0), put(0);
    for (int i = 0; i < steps; ++i) {
      __syncthreads();  // stage i is in place, and nobody reads the one before
      if (i + 1 < steps) fetch(i + 1);
      stage(i, std::false_type{});
      if (i + 1 < steps) put(i + 1);
    }
  }
  if constexpr (kApart) {
#pragma unroll
    for (int f = 0; f < MF; ++f)
#pragma unroll
      for (int s = 0; s < 4; ++s) acc[f][s] = total[f][s];
  }
}

// NS fragments of 16 columns of a wave's rows leave through its BYTES of LDS, so that
// lanes store consecutive bytes of a row of out: value(f, s, e) is column 4 * quad + e of
// fragment s (JOIN: 4 * NS * quad + 4 * s + e) in row `col` of fragment f.  to(row, c)
// says where the 16-byte piece c of the wave's row goes and how many of its elements (n
// <= 0: none), and whether as zeros.  The stores pass the caches by.
template <typename E>
struct Dst {
  E* p;
  int n;
  bool zero;
};
template <typename E, int MF, int NS, bool JOIN, int BYTES, typename V, typename T>
__device__ __forceinline__ void store_rows(uint8_t* mine, V value, T to) {
  constexpr int kRowBytes = 16 * NS * (int)sizeof(E), kPieces = kRowBytes / 16;
  constexpr int kPart = part_of(MF, BYTES / kRowBytes / 16);
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
  auto place = [&](int x, int c) {
    return mine + x * kRowBytes + 16 * (c ^ (x & (kPieces - 1) & 7));
  };
#pragma unroll
  for (int f0 = 0; f0 < MF; f0 += kPart) {
    wave_exchange();  // what was here has been read
#pragma unroll
    for (int f = f0; f < f0 + kPart; ++f)
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        Piece<E, 4> o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o.e[e] = from_f32<E>(value(f, s, e));
        const int byte = (JOIN ? 4 * NS * quad + 4 * s : 16 * s + 4 * quad) * (int)sizeof(E);
        __builtin_memcpy(place((f - f0) * 16 + col, byte / 16) + byte % 16, o.e, sizeof(o.e));
      }
    wave_exchange();
    constexpr int kPer = 64 / kPieces;  // rows of a store instruction
#pragma unroll
    for (int x0 = 0; x0 < kPart * 16; x0 += kPer) {
      const int x = x0 + lane / kPieces, c = lane % kPieces;
      const Dst<E> d = to(f0 * 16 + x, c);
      if (d.n <= 0) continue;
      Piece<E> o{};
      if (!d.zero) __builtin_memcpy(o.e, place(x, c), 16);
      if (d.n >= Piece<E>::kN)
        o.store_past(d.p);
      else
        o.store_head(d.p, d.n);
    }
  }
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
struct Live {
  uint8_t row[kMostRows];  // 1: computed, 2: set to zero, 0: left
};

// ONCE: these are all rows of their group, so b is read by this workgroup alone and passes
// the caches by (16384 rows over 166 groups, down: 610 us against 601).
template <typename E, bool ACROSS, bool GLU, int WA, int MF, int S, bool DMA, bool ONCE>
__device__ __forceinline__ void rows_tile(const RowsProduct& p, const Rows& r, int n0,
                                          uint8_t* smem, Live& live) {
  constexpr int kPiece = 16 / (int)sizeof(E);
  constexpr int kC = kStep / (int)sizeof(E);  // contraction steps of a stage
  constexpr bool JOIN = !ACROSS;              // a lane ends with consecutive columns
  constexpr int kOut = GLU ? 8 : 16;          // how many
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WA, wn = wave % WA;
  const E* b = (const E*)p.b + (size_t)r.g * p.b_group_stride;

  // the rows of a and (along) of b that the lane loads
  constexpr int kCols = Wide<WA>::kCols, kHalf = kCols / 2;
  constexpr int kLoadsL = 2 * MF / WA, kLoadsR = kCols / 16 / WA;  // 8 rows each
  const E* arow[kLoadsL];
#pragma unroll
  for (int j = 0; j < kLoadsL; ++j) {
    const int m = r.lo + (wave * kLoadsL + j) * 8 + (lane >> 3);
    arow[j] = (const E*)p.a + (size_t)max(source_row(p, min(m, r.hi - 1)), 0) * p.a_stride;
  }
  const E* brow[ACROSS ? 1 : kLoadsR];
  if constexpr (!ACROSS) {
    // row 64 w + 16 s + x of b in LDS is the row that gives lane quad q of the result the
    // columns kOut * q + 4 * s + i
#pragma unroll
    for (int j = 0; j < kLoadsR; ++j) {
      const int l = (wave * kLoadsR + j) * 8 + (lane >> 3);
      const int s = (l >> 4) & 3, x = l & 15;
      const int n = n0 + (l >> 6) * 4 * kOut + kOut * (x >> 2) + 4 * (GLU ? s & 1 : s) + (x & 3);
      brow[j] = b + (size_t)(min(n, p.N - 1) + (GLU && s >= 2 ? p.N : 0)) * p.b_stride;
    }
  }
  auto from_left = [&](int i, int j, int, int piece) {
    const int k = i * kC + piece * kPiece;
    return Src<E>{arow[j] + k, p.K - k};
  };
  auto from_right = [&](int i, int j, int row, int piece) {
    if constexpr (ACROSS) {
      const int k = i * kC + row, c = piece * kPiece;
      const int n = n0 + (GLU ? c % kHalf : c);
      return Src<E>{b + (size_t)k * p.b_stride + (GLU && c >= kHalf ? p.N : 0) + n,
                    k < p.K ? p.N - n : 0};
    } else {
      const int k = i * kC + piece * kPiece;
      return Src<E>{brow[j] + k, p.K - k};
    }
  };

  f32x4 acc[MF][4] = {};
  for (int t = threadIdx.x; t < 32 * MF; t += Wide<WA>::kThreads) {
    const bool in = r.lo + t < r.hi;
    live.row[t] = !in ? 0 : source_row(p, r.lo + t) >= 0 ? 1 : p.zero_rest ? 2 : 0;
  }
  products<E, false, ACROSS, GLU, WA, MF, S, DMA, ONCE>(
      smem, (p.K + kC - 1) / kC, [](int) {}, from_left, from_right, acc);
  barrier();  // every wave has read the last stage
  constexpr int kBytes = WA == kLarge ? 16384 : 8192;  // LDS that a wave's results pass through
  uint8_t* mine = smem + wave * kBytes;
  auto to = [&](auto* out, size_t stride, int at, int row, int c) {
    using O = std::remove_pointer_t<decltype(out)>;
    const int t = wm * MF * 16 + row, n = at + c * (16 / (int)sizeof(O));
    return Dst<O>{out + (size_t)(r.lo + t) * stride + n, live.row[t] ? p.N - n : 0,
                  live.row[t] == 2};
  };
  if constexpr (GLU) {
    const int n = n0 + wn * 32;
    if (p.pre) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        store_rows<float, MF, 2, JOIN, kBytes>(
            mine, [&](int f, int s, int e) { return acc[f][2 * h + s][e]; },
            [&](int row, int c) { return to(p.pre + (size_t)h * p.N, p.pre_stride, n, row, c); });
    }
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      float g[8], u[8], y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = acc[f][j / 4][j % 4], u[j] = acc[f][2 + j / 4][j % 4];
      swiglu(g, u, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[f][j / 4][j % 4] = y[j];
    }
  }
  auto leave = [&](auto* out) {
    store_rows<std::remove_pointer_t<decltype(out)>, MF, GLU ? 2 : 4, JOIN, kBytes>(
        mine, [&](int f, int s, int e) { return acc[f][s][e]; },
        [&](int row, int c) {
          return to(out, p.out_stride, n0 + wn * (GLU ? 32 : 64), row, c);
        });
  };
  if (p.out_f32)
    leave((float*)p.out);
  else
    leave((E*)p.out);
}

// Rows that nothing is computed for.
template <typename E>
__device__ __forceinline__ void zero_rows(const RowsProduct& p, const Rows& r, int n0, int n1) {
  if constexpr (sizeof(E) != 4)
    if (p.out_f32) return zero_rows<float>(p, r, n0, n1);
  void* out = p.out;
  const size_t stride = p.out_stride;
  constexpr int kPiece = 16 / (int)sizeof(E);
  const int pieces = (n1 - n0 + kPiece - 1) / kPiece;
  for (int t = threadIdx.x; t < (r.hi - r.lo) * pieces; t += blockDim.x) {
    const int n = n0 + t % pieces * kPiece;
    const Piece<E> o{};
    o.store_upto((E*)out + (size_t)(r.lo + t / pieces) * stride + n, n1 - n);
  }
}

// The rows of a workgroup, or the rest that it sets to zero.
template <typename E, int WA, bool GLU>
__device__ __forceinline__ bool tile_rows(const RowsProduct& p, int R, int64_t item, int n0,
                                          int* counts, Rows& r) {
  int64_t total = 0;
  if (find_rows(p, item, R, counts, r, total)) return true;
  constexpr int kWide = Wide<WA>::kCols / (GLU ? 2 : 1);
  if (p.zero_rest && rest_rows(p, item - total, R, r))
    zero_rows<E>(p, r, n0, min(n0 + kWide, p.N));
  return false;
}

template <typename E, bool ACROSS, bool GLU, bool DMA>
__global__ __launch_bounds__(Wide<kLarge>::kThreads, 2) void rows_tiles(RowsProduct p, int R,
                                                                       int cols, bool blocks,
                                                                       int64_t first) {
  constexpr int WA = kLarge;
  __shared__ __attribute__((aligned(1024))) uint8_t
      smem[2 * (kMostRows + Wide<WA>::kCols) * kStep];
  __shared__ Live live;
  __shared__ int counts[Wide<WA>::kWaves];
  int64_t item;
  int col;
  Rows r;
  tile_of(first + blockIdx.x, blocks, cols, item, col);
  if (col >= cols) return;
  const int n0 = col * (Wide<WA>::kCols / (GLU ? 2 : 1));
  if (!tile_rows<E, WA, GLU>(p, R, item, n0, counts, r)) return;
  const int rows = r.hi - r.lo;
  if constexpr (sizeof(E) == 4) {  // two sets of sums
    if (rows <= 64)
      rows_tile<E, ACROSS, GLU, WA, 2, 2, DMA, false>(p, r, n0, smem, live);
    else
      rows_tile<E, ACROSS, GLU, WA, 4, 2, DMA, false>(p, r, n0, smem, live);
  } else if constexpr (DMA) {
    if (rows <= 64 && r.all)
      rows_tile<E, ACROSS, GLU, WA, 2, 3, true, true>(p, r, n0, smem, live);
    else if (rows <= 64)
      rows_tile<E, ACROSS, GLU, WA, 2, 3, true, false>(p, r, n0, smem, live);
    else if (rows <= 128 && r.all)
      rows_tile<E, ACROSS, GLU, WA, 4, 3, true, true>(p, r, n0, smem, live);
    else if (rows <= 128)
      rows_tile<E, ACROSS, GLU, WA, 4, 3, true, false>(p, r, n0, smem, live);
    else if (rows <= 192)
      rows_tile<E, ACROSS, GLU, WA, 6, 2, true, false>(p, r, n0, smem, live);
    else if (rows <= 256)
      rows_tile<E, ACROSS, GLU, WA, 8, 2, true, false>(p, r, n0, smem, live);
    else
      rows_tile<E, ACROSS, GLU, WA, 10, 2, true, false>(p, r, n0, smem, live);
  } else {
    if (rows <= 64)
      rows_tile<E, ACROSS, GLU, WA, 2, 2, false, false>(p, r, n0, smem, live);
    else if (rows <= 128)
      rows_tile<E, ACROSS, GLU, WA, 4, 2, false, false>(p, r, n0, smem, live);
    else
      rows_tile<E, ACROSS, GLU, WA, 8, 2, false, false>(p, r, n0, smem, live);
  }
}

// Products of few tiles: 64 rows by 64 columns, two waves; with direct loads three stages
// ahead, since what each of the few workgroups has under way bounds them (4 rows over 8
// groups, K 4096, N 1024, b across: 58 us through registers, one stage ahead, against 33).
template <typename E, bool ACROSS, bool GLU, bool DMA>
__global__ __launch_bounds__(Wide<kSmall>::kThreads, 2) void rows_small(RowsProduct p, int cols,
                                                                       int64_t first) {
  constexpr int WA = kSmall, S = DMA ? 4 : 2;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * (64 + Wide<WA>::kCols) * kStep];
  __shared__ Live live;
  __shared__ int counts[Wide<WA>::kWaves];
  const int64_t id = first + blockIdx.x;
  const int n0 = (int)(id % cols) * (Wide<WA>::kCols / (GLU ? 2 : 1));
  Rows r;
  if (!tile_rows<E, WA, GLU>(p, 64, id / cols, n0, counts, r)) return;
  rows_tile<E, ACROSS, GLU, WA, 2, S, DMA, false>(p, r, n0, smem, live);
}

// Streaming form, for few rows in few groups, b along its rows: a workgroup takes 32 rows of b
// (with SwiGLU, 16 gate rows and their 16 up rows) and up to 16 rows of one group, its
// waves each a run of K; the sums are added through LDS in a fixed order.  b goes from
// memory straight to the registers of the matrix instruction (lane l: row l % 16, bytes 16
// (l / 16) of 64), from any address, kAhead steps before its products.
constexpr int kSWaves = 8;

template <typename E, bool GLU>
__global__ __launch_bounds__(kSWaves* kWave) void rows_stream(RowsProduct p, int cols,
                                                             int64_t first) {
  constexpr int kPiece = 16 / (int)sizeof(E), kC = kStep / (int)sizeof(E);
  constexpr int kRing = 4, kAhead = kRing - 1;
  __shared__ f32x4 part[kSWaves][2][kWave];
  __shared__ int counts[kSWaves];
  const int64_t id = first + blockIdx.x;
  const int n0 = (int)(id % cols) * (GLU ? 16 : 32);
  Rows r;
  int64_t total = 0;
  if (!find_rows(p, id / cols, 16, counts, r, total)) {
    if (p.zero_rest && rest_rows(p, id / cols - total, 16, r))
      zero_rows<E>(p, r, n0, min(n0 + (GLU ? 16 : 32), p.N));
    return;
  }
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int col = lane & 15, quad = lane >> 4;
  const E* b = (const E*)p.b + (size_t)r.g * p.b_group_stride + kPiece * quad;
  const E* row[3];  // two of b, one of a
  row[0] = b + (size_t)min(n0 + col, p.N - 1) * p.b_stride;
  row[1] = b + (size_t)(GLU ? p.N + min(n0 + col, p.N - 1) : min(n0 + 16 + col, p.N - 1)) *
                   p.b_stride;
  const int src = source_row(p, min(r.lo + col, r.hi - 1));
  row[2] = (const E*)p.a + (size_t)max(src, 0) * p.a_stride + kPiece * quad;

  struct Step {
    i32x4 v[3][2];
  };
  auto load = [&](Step& w, int c) {
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w.v[s][h] = __builtin_bit_cast(i32x4, *(const u32x4*)(row[s] + c * kC + h * (kC / 2)));
  };
  f32x4 acc[2] = {};
  auto multiply = [&](const Step& w) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int s = 0; s < 2; ++s) acc[s] = mma<E>(w.v[s][h], w.v[2][h], acc[s]);
  };
  // the wave's whole steps [lo, hi); loads past its last repeat that one
  const int full = p.K / kC;
  const int lo = (int)((int64_t)full * wave / kSWaves);
  const int hi = (int)((int64_t)full * (wave + 1) / kSWaves);
  if (lo < hi) {
    Step w[kRing];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load(w[u], min(lo + u, hi - 1));
    for (int c0 = lo; c0 < hi; c0 += kRing) {
#pragma unroll
      for (int u = 0; u < kRing; ++u) {
        if (c0 + u >= hi) break;
        load(w[(u + kAhead) % kRing], min(c0 + u + kAhead, hi - 1));
        multiply(w[u]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if (p.K % kC && wave == kSWaves - 1) {  // what the end of the rows leaves of a step
    Step w;
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = full * kC + h * (kC / 2), n = p.K - k - kPiece * quad;
        Piece<E> u{};
        if (n > 0) u.load_upto(row[s] + k, n);
        __builtin_memcpy(&w.v[s][h], u.e, 16);
      }
    multiply(w);
  }

#pragma unroll
  for (int s = 0; s < 2; ++s) part[wave][s][lane] = acc[s];
  __syncthreads();
  // lane: row `col` of out, columns 4 * quad .. + 3 of each 16
  const int m = r.lo + col, n = n0 + 4 * quad;
  const bool live = m < r.hi && src >= 0;
  if (wave > 0 || m >= r.hi || !(live || p.zero_rest)) return;
  f32x4 sum[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    sum[s] = part[0][s][lane];
#pragma unroll
    for (int w = 1; w < kSWaves; ++w) sum[s] += part[w][s][lane];
  }
  auto store = [&](auto* out, size_t stride, int at, const float (&y)[4]) {
    using O = std::remove_pointer_t<decltype(out)>;
    Piece<O, 4> o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.e[i] = from_f32<O>(live ? y[i] : 0.0f);
    if (at < p.N) o.store_upto(out + (size_t)m * stride + at, p.N - at);
  };
  float y[2][4];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) y[s][i] = sum[s][i];
  if constexpr (GLU) {
    if (p.pre) {
      store(p.pre, p.pre_stride, n, y[0]);
      store(p.pre + p.N, p.pre_stride, n, y[1]);
    }
    float h[4];
    swiglu(y[0], y[1], h);
    if (p.out_f32)
      store((float*)p.out, p.out_stride, n, h);
    else
      store((E*)p.out, p.out_stride, n, h);
  } else {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (p.out_f32)
        store((float*)p.out, p.out_stride, n + 16 * s, y[s]);
      else
        store((E*)p.out, p.out_stride, n + 16 * s, y[s]);
    }
  }
}

// Most rows of a tile: more rows share a load of b's, but a product of few tiles may
// then leave more of the 256 CUs without one; its time goes as rounds * (rows + 256).
inline int rows_of_tile(int M, int G, int cols, int most) {
  const int64_t groups = G < M ? G : M;
  if ((M / most + groups) * cols >= 256) return most;
  int best = most;
  int64_t least = INT64_MAX;
  for (int R : {320, 256, 192, 128, 64}) {
    if (R > most) continue;
    const int64_t cost = ((M / R + groups) * cols + 255) / 256 * (R + 256);
    if (cost < least) best = R, least = cost;
  }
  return best;
}

// Below so many tiles, of 64 rows even, most of the 256 CUs would be left without one: then
// 64 x 64 tiles, or with few rows in each group the streaming form (8 groups of one row, K
// 4096, 2N 4096: 51 us, 5.2 TB/s; at 16 groups, 256 tiles, it takes 100 where tiles take 81).
constexpr int kFewTiles = 192;

template <typename E, bool ACROSS, bool GLU>
void launch_rows_tiles(const RowsProduct& p, bool dma, hipStream_t stream) {
  constexpr int per = Wide<kLarge>::kCols / (GLU ? 2 : 1);
  const int cols = (p.N + per - 1) / per;
  const int64_t groups = p.G < p.M ? p.G : p.M, few = (p.M / 64 + groups) * cols;
  if constexpr (!ACROSS) {
    if (few < kFewTiles && (p.M <= 16 || p.M < 4 * groups)) {
      const int scols = (p.N + (GLU ? 15 : 31)) / (GLU ? 16 : 32);
      const int64_t all = (max_items(p.M, p.G, 16) + (p.zero_rest ? 2 : 0)) * scols;
      for (int64_t first = 0; first < all; first += kMaxGrid) {
        const unsigned grid = (unsigned)(all - first < kMaxGrid ? all - first : kMaxGrid);
        rows_stream<E, GLU><<<grid, kSWaves * kWave, 0, stream>>>(p, scols, first);
      }
      return;
    }
  }
  if (few < kFewTiles) {
    constexpr int small = Wide<kSmall>::kCols / (GLU ? 2 : 1);
    const int scols = (p.N + small - 1) / small;
    const int64_t all = (max_items(p.M, p.G, 64) + (p.zero_rest ? 2 : 0)) * scols;
    for (int64_t first = 0; first < all; first += kMaxGrid) {
      const unsigned grid = (unsigned)(all - first < kMaxGrid ? all - first : kMaxGrid);
      if (dma)
        rows_small<E, ACROSS, GLU, true><<<grid, Wide<kSmall>::kThreads, 0, stream>>>(p, scols, first);
      else
        rows_small<E, ACROSS, GLU, false><<<grid, Wide<kSmall>::kThreads, 0, stream>>>(p, scols, first);
    }
    return;
  }
  const int R = rows_of_tile(p.M, p.G, cols, sizeof(E) == 4 ? 128 : dma ? kMostRows : 256);
  const int64_t items = max_items(p.M, p.G, R) + (p.zero_rest ? 2 : 0);
  const bool blocks = p.M > 128 * (int64_t)p.G && items * cols >= 2048;
  const int64_t tiles =
      blocks ? (int64_t)up_to((items + kBlockItems - 1) / kBlockItems *
                                  ((cols + kBlockCols - 1) / kBlockCols), 8) *
                   kBlockItems * kBlockCols
             : items * cols;
  for (int64_t first = 0; first < tiles; first += kMaxGrid) {
    const unsigned grid = (unsigned)(tiles - first < kMaxGrid ? tiles - first : kMaxGrid);
    if (dma)
      rows_tiles<E, ACROSS, GLU, true><<<grid, Wide<kLarge>::kThreads, 0, stream>>>(p, R, cols, blocks, first);
    else
      rows_tiles<E, ACROSS, GLU, false><<<grid, Wide<kLarge>::kThreads, 0, stream>>>(p, R, cols, blocks, first);
  }
}

// Whether rows of n elements, `stride` apart, consist of whole 16-byte pieces.
template <typename E>
inline bool whole_pieces(const void* p, size_t stride, size_t group_stride, int n) {
  constexpr size_t kPiece = 16 / sizeof(E);
  return aligned(p, 16) && stride % kPiece == 0 && group_stride % kPiece == 0 && n % kPiece == 0;
}

template <typename E>
int launch_rows_product(const RowsProduct& p, bool across, bool glu, hipStream_t stream) {
  const bool dma = whole_pieces<E>(p.a, p.a_stride, 0, p.K) &&
                   whole_pieces<E>(p.b, p.b_stride, p.b_group_stride, across ? p.N : p.K);
  if (across && glu)
    launch_rows_tiles<E, true, true>(p, dma, stream);
  else if (across)
    launch_rows_tiles<E, true, false>(p, dma, stream);
  else if (glu)
    launch_rows_tiles<E, false, true>(p, dma, stream);
  else
    launch_rows_tiles<E, false, false>(p, dma, stream);
  return hip_status();
}

// ---------------------------------------------------------------------------
// outer
// ---------------------------------------------------------------------------
// Rows of an indexed operand are looked up once, into a table in LDS: of kTable rows of
// the group at a time, each with a run of the main loop of its own.  (An index read from
// memory ahead of each load: 64 groups of 512 rows, 4096 x 4096, 3086 us.)
constexpr int kTable = 2048;
enum { kNone, kLeft, kRight };  // the operand that has an index

template <typename E, int WA, int MF, bool DMA, int INDEXED>
__global__ __launch_bounds__(Wide<WA>::kThreads, 2) void outer_tiles(OuterProduct p, int down,
                                                                    int across, bool blocks,
                                                                    int64_t first) {
  constexpr int kRows = 32 * MF, kCols = Wide<WA>::kCols, kThreads = Wide<WA>::kThreads;
  constexpr int kPiece = 16 / (int)sizeof(E);
  constexpr int kC = kStep / (int)sizeof(E);
  constexpr int kLoads = 2 * MF / WA;  // of each operand
  static_assert(kRows == kCols, "both operands' loads take the same rows");
  constexpr int kBytes = 2 * (kRows + kCols) * kStep;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kBytes];
  __shared__ int table[INDEXED == kNone ? 1 : kTable];
  int64_t item;
  int col;
  tile_of(first + blockIdx.x, blocks, across, item, col);
  const int64_t group = item / down;
  if (col >= across || group >= p.G) return;
  const int g = (int)group, l0 = (int)(item % down) * kRows, r0 = col * kCols;
  int lo = clamp_row(p.offsets[g], p.M), hi = clamp_row(p.offsets[g + 1], p.M);
  if (p.sums && hi > lo) {
    const int part = ((hi - lo + p.splits - 1) / p.splits + kC - 1) / kC * kC;
    lo = (int)min((int64_t)hi, lo + (int64_t)blockIdx.y * part);
    hi = min(hi, lo + part);
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WA, wn = wave % WA;

  f32x4 acc[MF][4] = {};
  constexpr int kRun = INDEXED == kNone ? 1 << 30 : kTable;
  for (int m0 = lo; m0 < hi; m0 += kRun) {
    const int n = min(hi - m0, kRun);
    if constexpr (INDEXED != kNone) {
      __syncthreads();  // the table and the last stage of the run before have been read
      const int32_t* index = INDEXED == kLeft ? p.left_index : p.right_index;
      const int div = INDEXED == kLeft ? p.left_div : p.right_div;
      const int rows = INDEXED == kLeft ? p.left_rows : p.right_rows;
      for (int t = threadIdx.x; t < n; t += kThreads) {
        int r = named_at(index, p.pos, p.M, m0 + t);
        r = r < 0 ? -1 : r / div;
        table[t] = (unsigned)r < (unsigned)rows ? r : -1;
      }
      __syncthreads();
    }
    int row_of[kLoads];  // of the indexed operand, for each load of a stage
    auto before = [&](int i) {
      if constexpr (INDEXED != kNone) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const int row =
              i * kC + ((wave * kLoads + j) * 64 + (int)(threadIdx.x & 63)) / (kCols / kPiece);
          row_of[j] = row < n ? table[row] : -1;
        }
      }
    };
    // both operands' loads j take the same rows, and a row that one lacks adds nothing
    auto from_left = [&](int i, int j, int row, int piece) {
      const int t = i * kC + row, c = l0 + piece * kPiece;
      const bool in = INDEXED == kNone ? t < n : row_of[j] >= 0;
      const int r = INDEXED == kLeft ? row_of[j] : m0 + t;
      return Src<E>{(const E*)p.left + (size_t)r * p.left_stride + c, in ? p.L - c : 0};
    };
    auto from_right = [&](int i, int j, int row, int piece) {
      const int t = i * kC + row, c = r0 + piece * kPiece;
      const bool in = INDEXED == kNone ? t < n : row_of[j] >= 0;
      const int r = INDEXED == kRight ? row_of[j] : m0 + t;
      return Src<E>{(const E*)p.right + (size_t)r * p.right_stride + c, in ? p.R - c : 0};
    };
    products<E, true, true, false, WA, MF, 2, DMA, false>(smem, (n + kC - 1) / kC, before, from_left,
                                                      from_right, acc);
  }
  barrier();
  constexpr int kMine = kBytes / Wide<WA>::kWaves;
  auto leave = [&](auto* to, size_t stride) {
    using O = std::remove_pointer_t<decltype(to)>;
    store_rows<O, MF, 4, false, kMine>(
        smem + wave * kMine, [&](int f, int s, int e) { return acc[f][s][e]; },
        [&](int row, int c) {
          const int l = l0 + wm * MF * 16 + row;
          const int n = r0 + wn * 64 + c * (16 / (int)sizeof(O));
          return Dst<O>{to + (size_t)l * stride + n, l < p.L ? p.R - n : 0, false};
        });
  };
  if constexpr (WA == kSmall)
    if (p.sums)
      return leave(p.sums + ((size_t)blockIdx.y * p.G + g) * ((size_t)p.L * p.R), (size_t)p.R);
  leave((E*)p.out + (size_t)g * p.out_group_stride, p.out_stride);
}

// The parts' sums, in order, rounded once.
template <typename E>
__global__ __launch_bounds__(256) void outer_sum(OuterProduct p) {
  const int64_t all = (int64_t)p.G * p.L * p.R;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    float v = p.sums[i];
    for (int s = 1; s < p.splits; ++s) v += p.sums[s * all + i];
    const int64_t row = i / p.R;
    ((E*)p.out)[(size_t)(row / p.L) * p.out_group_stride + (size_t)(row % p.L) * p.out_stride +
                (size_t)(i % p.R)] = from_f32<E>(v);
  }
}

// Tiles of n x n, whether they are few, and into how many parts a group's rows are then cut:
// enough for two workgroups a CU, of 512 rows at least, counted for groups of equal sizes (two
// groups of 16384 rows, 256 x 192: 24 tiles).  Few are counted without the rows, so moderate
// matrices over many rows take the small tiles too (eight groups of 1024 x 1024: 128 large ones).
inline int64_t outer_tiles_of(int L, int R, int G, int n) {
  return (int64_t)G * ((L + n - 1) / n) * ((R + n - 1) / n);
}
inline bool few_outer_tiles(int L, int R, int G, int dtype) {
  return outer_tiles_of(L, R, G, 64 * (dtype == MOE_DT_FP32 ? kOuter<float> : kOuter<Bf16>)) <
         kFewTiles;
}
inline int outer_splits(int M, int L, int R, int G, int dtype) {
  if (!few_outer_tiles(L, R, G, dtype)) return 1;
  const int64_t want = 512 / outer_tiles_of(L, R, G, 64), most = M / (512 * (int64_t)G);
  const int64_t n = want < most ? want : most;
  return n < 2 ? 1 : n > 64 ? 64 : (int)n;
}


template <typename E, int INDEXED>
void launch_outer_tiles(const OuterProduct& p, hipStream_t stream) {
  const bool dma = whole_pieces<E>(p.left, p.left_stride, 0, p.L) &&
                   whole_pieces<E>(p.right, p.right_stride, 0, p.R);
  constexpr int WA = kOuter<E>;
  auto tiles_of = [&](int n) { return outer_tiles_of(p.L, p.R, p.G, n); };
  const bool few = tiles_of(64 * WA) < kFewTiles;
  const int side = few ? 64 : 64 * WA, down = (p.L + side - 1) / side, across = (p.R + side - 1) / side;
  // Blocks of tiles for each XCD, whose L2 then serves each operand's columns several times,
  // pay where there are many tiles of many rows (64 groups of 512 rows, 4096 x 4096: 1424 us
  // against 1367), and cost where there are fewer (32 of 460, 2048 x 4096: 296 against 311) or
  // only zeros are written (230 groups without rows: 1190 against 1300).
  const bool blocks = tiles_of(side) >= 8192 && p.M >= 256 * (int64_t)p.G;
  const int64_t items = (int64_t)p.G * down;
  const int64_t tiles =
      blocks ? (int64_t)up_to((items + kBlockItems - 1) / kBlockItems *
                                  ((across + kBlockCols - 1) / kBlockCols), 8) *
                   kBlockItems * kBlockCols
             : items * across;
  for (int64_t first = 0; first < tiles; first += kMaxGrid) {
    const unsigned grid = (unsigned)(tiles - first < kMaxGrid ? tiles - first : kMaxGrid);
    if (few)
      outer_tiles<E, kSmall, 2, false, INDEXED>
          <<<dim3(grid, p.sums ? p.splits : 1), Wide<kSmall>::kThreads, 0, stream>>>(p, down, across, blocks, first);
    else if (dma)
      outer_tiles<E, WA, 2 * WA, true, INDEXED>
          <<<grid, Wide<WA>::kThreads, 0, stream>>>(p, down, across, blocks, first);
    else
      outer_tiles<E, WA, 2 * WA, false, INDEXED>
          <<<grid, Wide<WA>::kThreads, 0, stream>>>(p, down, across, blocks, first);
  }
  if (p.sums) {
    const int64_t want = ((int64_t)p.G * p.L * p.R + 255) / 256;
    outer_sum<E><<<(unsigned)(want < 4096 ? want : 4096), 256, 0, stream>>>(p);
  }
}

template <typename E>
int launch_outer_product(const OuterProduct& p, hipStream_t stream) {
  if (p.left_index)
    launch_outer_tiles<E, kLeft>(p, stream);
  else if (p.right_index)
    launch_outer_tiles<E, kRight>(p, stream);
  else
    launch_outer_tiles<E, kNone>(p, stream);
  return hip_status();
}

}  // namespace moe
