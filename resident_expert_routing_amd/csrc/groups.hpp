// What the products over a bucketing share: which rows of which group a workgroup
// has, the row of the input that a row of the output names, SwiGLU, and the tiled
// forms' loads, waits and order of tiles.  Arguments P have M, G, offsets; source_row
// also index, index_div, a_rows.
#pragma once

#include "elements.hpp"

namespace moe {

constexpr int kMaxGrid = 1 << 22;  // workgroups of a launch

struct Rows {
  int g, lo, hi;  // rows [lo, hi) of out, at most as many as asked for, of group g
  bool all;       // the group has no others
};

__device__ __forceinline__ int clamp_row(int v, int M) { return min(max(v, 0), M); }

// Which rows a workgroup has.  The groups' rows are cut into pieces of at most R,
// counted through the groups in order, and the workgroup finds the item-th piece
// by itself.  A wave looks at 256 groups at a time, a lane at four: a scan over
// the lanes gives the sums of their pieces, and the first lane whose sum passes
// `item` holds its group.  More groups (an arena of many layers) are first counted
// by all waves, each a run of them, side by side: with every wave walking all of
// them a lane's loads followed one another, 8 rows over 1000 groups took 39 us
// against 32, 256 over 6666 groups 79 against 27.  Offsets outside [0, M] are cut,
// and sums stop at a bound above every count, so that offsets which are no
// bucketing cannot overflow them.
constexpr int kShare = 4;            // groups of a lane
constexpr int kChunk = 64 * kShare;  // groups of a wave at a time
constexpr int kMostPieces = 1 << 29;

__device__ __forceinline__ int pieces_of(int lo, int hi, int R) {
  return hi > lo ? (hi - lo) / R + ((hi - lo) % R != 0) : 0;
}

// Inclusive sums over the lanes: within rows of 16, then lane 15 of a row into
// the next, then lane 31 into the upper half.
__device__ __forceinline__ int wave_scan(int v) {
#define MOE_SCAN_STEP(CTRL, ROWS) \
  v = min(v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false), kMostPieces);
  MOE_SCAN_STEP(0x111, 0xF)  // row_shr by 1, 2, 4, 8
  MOE_SCAN_STEP(0x112, 0xF)
  MOE_SCAN_STEP(0x114, 0xF)
  MOE_SCAN_STEP(0x118, 0xF)
  MOE_SCAN_STEP(kDppBcast15, 0xA)
  MOE_SCAN_STEP(kDppBcast31, 0xC)
#undef MOE_SCAN_STEP
  return v;
}

// The offsets of this lane's groups of the chunk from group `base` on, and the
// pieces of all groups up to and with the lane's.
template <typename P>
__device__ __forceinline__ int chunk_sums(const P& p, int base, int R,
                                          int (&edge)[kShare + 1]) {
  const int g = base + (threadIdx.x & 63) * kShare;
#pragma unroll
  for (int i = 0; i <= kShare; ++i) edge[i] = clamp_row(p.offsets[min(g + i, p.G)], p.M);
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kShare; ++i) mine += pieces_of(edge[i], edge[i + 1], R);
  return wave_scan(min(mine, kMostPieces));
}

// Piece `item` of the chunk; returns the chunk's pieces, and sets r if there are
// more than item.
template <typename P>
__device__ __forceinline__ int piece_of_chunk(const P& p, int base, int R, int item,
                                              Rows& r) {
  int edge[kShare + 1];
  const int lane = threadIdx.x & 63, sum = chunk_sums(p, base, R, edge);
  const int total = __builtin_amdgcn_readlane(sum, 63);
  if (item >= total) return total;
  const int owner = __ffsll((long long)__ballot(sum > item)) - 1;
  const int before = __shfl_up(sum, 1, 64);
  int i = 0, left = item - (lane == 0 ? 0 : before), lo = edge[0], hi = edge[1];
#pragma unroll
  for (int j = 1; j < kShare; ++j) {  // left: of the pieces from group i on
    const int n = pieces_of(lo, hi, R);
    if (i == j - 1 && left >= n) i = j, left -= n, lo = edge[j], hi = edge[j + 1];
  }
  lo = __builtin_amdgcn_readlane(lo, owner);
  hi = __builtin_amdgcn_readlane(hi, owner);
  r.g = base + owner * kShare + __builtin_amdgcn_readlane(i, owner);
  r.lo = lo + __builtin_amdgcn_readlane(left, owner) * R;
  r.hi = r.lo + min(R, hi - r.lo);
  r.all = hi - lo <= R;
  return total;
}

// The workgroup's rows; false if there are not that many pieces, `total` then says how
// many.  Reached by all its waves; `counts` is an LDS word for each.
template <typename P>
__device__ __forceinline__ bool find_rows(const P& p, int64_t item, int R, int* counts, Rows& r,
                                          int64_t& total) {
  if (!p.offsets) {
    total = pieces_of(0, p.M, R);
    if (item >= total) return false;
    const int lo = (int)item * R;
    r = {0, lo, lo + min(R, p.M - lo), p.M <= R};
    return true;
  }
  if (p.G <= kChunk) {
    total = piece_of_chunk(p, 0, R, (int)(item < kMostPieces ? item : kMostPieces), r);
    return item < total;
  }
  const int chunks = (p.G + kChunk - 1) / kChunk, waves = blockDim.x / kWave;
  const int run = (chunks + waves - 1) / waves, wave = threadIdx.x / kWave;
  int mine = 0;
  for (int c = wave * run; c < min(wave * run + run, chunks); ++c) {
    int edge[kShare + 1];
    const int sum = __builtin_amdgcn_readlane(chunk_sums(p, c * kChunk, R, edge), 63);
    mine = min(mine + sum, kMostPieces);
  }
  if ((threadIdx.x & 63) == 0) counts[wave] = mine;
  __syncthreads();
  int64_t before = 0;
  int w = 0;
  while (w < waves && item >= before + counts[w]) before += counts[w++];
  for (int c = w * run; c < min(w * run + run, chunks); ++c) {
    const int64_t left = item - before;
    const int n = piece_of_chunk(p, c * kChunk, R, (int)(left < kMostPieces ? left : kMostPieces), r);
    if (left < n) return true;
    before += n;
  }
  total = before;
  return false;
}
template <typename P>
__device__ __forceinline__ bool find_rows(const P& p, int64_t item, int R, int* counts, Rows& r) {
  int64_t total = 0;
  return find_rows(p, item, R, counts, r, total);
}

// Piece `item` of the rows in no group (before the first and behind the last), for calls
// that zero them: at most max_items(M, 0, R) + 1 pieces.
template <typename P>
__device__ __forceinline__ bool rest_rows(const P& p, int64_t item, int R, Rows& r) {
  const int first = clamp_row(p.offsets[0], p.M), last = max(first, clamp_row(p.offsets[p.G], p.M));
  const int head = pieces_of(0, first, R);
  const int64_t lo = item < head ? item * R : last + (item - head) * R;
  const int end = item < head ? first : p.M;
  if (lo >= end) return false;
  r = {0, (int)lo, (int)min(lo + R, (int64_t)end), false};
  return true;
}

// Most pieces of R rows that M rows in G groups can make.
inline int64_t max_items(int M, int G, int R) {
  return (int64_t)M / R + (G > 0 ? (G < M ? G : M) : 1);
}

// The row of a that row m of out is computed from; -1 if it names none.
template <typename P>
__device__ __forceinline__ int source_row(const P& p, int m) {
  int r = m;
  if (p.index) {
    r = p.index[m];
    r = r < 0 ? -1 : r / p.index_div;
  }
  return (unsigned)r < (unsigned)p.a_rows ? r : -1;
}

// silu(g) * u, silu(g) = g / (1 + exp(-g)), of N values.  The reciprocal's error is
// one unit in the last place, where the division's ten instructions took 2 us of
// a tile's epilogue; exp(-g) = 2^(-g log2 e), whose rounded argument is off by
// |g| * 1.25 * 2^-24 of the result, is within two units more.  From -88 down exp
// overflows, and the product would be zero where the value is still a normal
// number: below kLow, where 1 + exp(-g) is exp(-g) in float32, the value is
// (g h) (h u) with h = exp(g / 2), so that only the result can be subnormal (h is
// down to g = -174).  Few gates get there: one minimum a value, one branch for N.
template <int N>
__device__ __forceinline__ void swiglu(const float (&g)[N], const float (&u)[N], float (&y)[N]) {
  constexpr float kLow = -64.0f;
  float least = g[0];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    least = fminf(least, g[i]);
    y[i] = g[i] * __builtin_amdgcn_rcpf(1.0f + __expf(-g[i])) * u[i];
  }
  if (__builtin_expect(least < kLow, 0)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float h = __expf(0.5f * g[i]);
      if (g[i] < kLow) y[i] = (g[i] * h) * (h * u[i]);
    }
  }
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// The wave's own LDS reads and writes are done when it arrives.
__device__ __forceinline__ void barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Lanes of a wave hand values to each other through LDS across this: LDS is in order
// within a wave, so the hardware waits for nothing, and the compiler is kept from
// moving accesses over it.
__device__ __forceinline__ void wave_exchange() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __align__(16) const uint8_t kZeros[16] = {};  // source of what lies behind a row

constexpr int part_of(int n, int most) {  // the largest divisor of n that is at most `most`
  int d = n < most ? n : most;
  while (n % d) --d;
  return d;
}

// dma16 past the caches (with its wait state), for bytes that no other workgroup
// reads.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is written here on purpose
__device__ __forceinline__ void dma16_past(const uint8_t* g, uint8_t* lds_base) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_u8*)lds_base);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt"
               :
               : "s"(m0), "v"(g)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// Which tile, item by column, workgroup `id` has.  Consecutive workgroups go to
// the 8 XCDs in turn.  With `blocks` an XCD gets blocks of kBlockItems x
// kBlockCols tiles, as many as it has CUs, so that its L2 serves each row of a and
// b several times; otherwise the columns of an item follow one another.
constexpr int kBlockItems = 8, kBlockCols = 4;

__device__ __forceinline__ void tile_of(int64_t id, bool blocks, int cols, int64_t& item,
                                        int& col) {
  if (blocks) {
    constexpr int kBlock = kBlockItems * kBlockCols;
    const int64_t j = id >> 3, block = (j / kBlock) * 8 + (id & 7);
    const int at = (int)(j % kBlock), across = (cols + kBlockCols - 1) / kBlockCols;
    item = block / across * kBlockItems + at / kBlockCols;
    col = (int)(block % across) * kBlockCols + at % kBlockCols;
  } else {
    item = id / cols, col = (int)(id % cols);
  }
}

}  // namespace moe
