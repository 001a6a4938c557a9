// Token rows in the order of the slots and back, with weights and gradients:
// moe_positions, moe_dispatch, moe_dispatch_backward, moe_combine,
// moe_combine_backward.
//
// With a = t*k + j the assignments and pos[a] the row that holds assignment a:
//   spread   row[pos[a]] = w[a] * token[t]                (dispatch; combine's backward)
//   gather   token[t]    = sum_j w[t,j] * row[pos[t,j]]   (combine; dispatch's backward)
// and the weight's gradient is the dot product of the row with the token row
// on the other side.  So two kernel forms serve all four calls.  All of them
// are token-major: a token row is read or written once while its k rows pass (a
// row-major dispatch, each row fetching its token's, was correct and slower: 8192
// tokens of 6144, top-8, 231 us against 183).  Sums run over ascending j in
// float32 in one thread, dot products in a fixed tree: no atomics, the same
// result on every call.
//
// All are bound by memory.  For 8192 tokens of 6144 bf16, top-8 (65536 rows, 805
// MB): spread 182 us (906 MB, 5.0 TB/s), gather 156 us (5.8 TB/s), spread with
// dot products 342 us (1.7 GB, 5.0 TB/s).  A copy of 1 GiB runs at 4.7 to 5.1 TB/s.
// Two times "A against B" below are of one form against the other when that choice
// was made.  Small calls are bound by dependent loads, a token's picks one after
// another: 32 tokens of 4096, top-8, spread 5.2 us, 8 tokens gather 4.0.
#include "elements.hpp"

using namespace moe;

namespace {

constexpr int kThreads = 512;
constexpr int kDotThreads = 256;
constexpr int kMaxGrid = 1 << 21;      // workgroups of a launch; they stride over the rest
constexpr int kLdsPositions = 4096;    // assignments that one workgroup orders in LDS

struct RowsArgs {
  int T, H, k, n;  // n = T*k rows
  const int32_t* perm;
  const int32_t* pos;
  const float* weight;
  const char* src;
  char* dst;
  const char* other;
  float* dweight;
  size_t src_stride, dst_stride, other_stride;  // bytes
};

// A workgroup has one token at a time, so its rows and weights are scalars and
// a row's address is a scalar base and a thread's 32-bit offset (H * 4 <= 2^32).
// Tokens are counted without a sign: the step of the grid leads past 2^31 - 1
// behind the last one of a batch of nearly as many.

// The rows of picks j0 .. j0 + 7 of token t: -1 past k and for absent ones.
__device__ __forceinline__ void rows_of(const RowsArgs& p, uint32_t t, int j0, int (&row)[8]) {
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    int r = -1;
    if (j0 + u < p.k) r = p.pos[(size_t)t * p.k + j0 + u];
    row[u] = __builtin_amdgcn_readfirstlane((unsigned)r < (unsigned)p.n ? r : -1);
  }
}

__device__ __forceinline__ void weights_of(const RowsArgs& p, uint32_t t, int j0, float (&w)[8]) {
#pragma unroll
  for (int u = 0; u < 8; ++u)
    w[u] = p.weight && j0 + u < p.k ? p.weight[(size_t)t * p.k + j0 + u] : 1.0f;
}

// A row is taken in pieces of N elements (16 bytes; single elements where the
// row has fewer).  The last piece of a row that N does not divide starts early,
// at H - N: what it shares with the piece before is computed twice, alike.
template <typename E, int N>
__device__ __forceinline__ uint32_t start_of(uint32_t i, uint32_t H) {
  return N == 1 ? i : min(i, H - N);
}
template <typename E, int N>
__device__ __forceinline__ void load_piece(Piece<E, N>& v, const char* row, uint32_t i) {
  v.load((const E*)(row + i * (uint32_t)sizeof(E)));
}

// Rows that are read once, T*k of them, pass the caches by (non-temporal), which
// leaves these to the token rows: combine of 65536 x 6144 bf16 rows 211 us
// against 167, with its gradient 772 against 547.
template <typename E, int N>
__device__ __forceinline__ void load_once(Piece<E, N>& v, const char* row, uint32_t i) {
  if constexpr (N * sizeof(E) == 16)
    v.load_past((const E*)(row + i * (uint32_t)sizeof(E)));
  else
    load_piece(v, row, i);
}

// NT: past the caches.  Beside such loads that is faster (the same combine 167
// us against 161, with its gradient 547 against 519), alone it is not (dispatch to
// those rows 181 us against 190).
template <bool NT, typename E, int N>
__device__ __forceinline__ void store_piece(const Piece<E, N>& v, char* row, uint32_t i) {
  if constexpr (NT && N * sizeof(E) == 16)
    v.store_past((E*)(row + i * (uint32_t)sizeof(E)));
  else
    v.store((E*)(row + i * (uint32_t)sizeof(E)));
}

template <typename E, int N>
__device__ __forceinline__ Piece<E, N> scaled(const Piece<E, N>& v, float w) {
  Piece<E, N> o;
#pragma unroll
  for (int i = 0; i < N; ++i) o.e[i] = from_f32<E>(w * to_f32<E>(v.e[i]));
  return o;
}

// The rows that belong to no assignment: those to which perm gives none (picks
// with no slot have no row of their own, so these are the last rows), and the
// earlier ones of an assignment that perm names twice, whose row is pos[a].  They
// are set to zero (row t*k + j by the workgroups of token t, the pieces from i0 to
// before i1 by this one).  Eight rows at a time, so that their loads overlap.
template <typename E, int N>
__device__ __forceinline__ void zero_unnamed(const RowsArgs& p, uint32_t t, uint32_t i0,
                                             uint32_t i1) {
  if (!p.perm) return;
  const size_t first = (size_t)t * p.k;
  for (int j0 = 0; j0 < p.k; j0 += 8) {
    int a[8], at[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) a[u] = p.perm[first + min(j0 + u, p.k - 1)];
#pragma unroll
    for (int u = 0; u < 8; ++u) at[u] = p.pos[(unsigned)a[u] < (unsigned)p.n ? a[u] : 0];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const size_t r = first + j0 + u;
      if (j0 + u >= p.k || ((unsigned)a[u] < (unsigned)p.n && at[u] == (int)r)) continue;
      for (uint32_t i = i0 + threadIdx.x * N; i < i1; i += blockDim.x * N)
        store_piece<false>(Piece<E, N>{}, p.dst + r * p.dst_stride, start_of<E, N>(i, p.H));
    }
  }
}

// spread: a thread reads pieces of a token row and stores each k times.  Bound
// by the stores, which are as many bytes as the rows have.  A workgroup holds up
// to kHold pieces a thread, so that it writes whole stretches of one row after
// another.
constexpr int kHold = 4;

template <typename E, int N, bool WEIGHT, bool NT>
__device__ __forceinline__ void spread_span(const RowsArgs& p, uint32_t t, uint32_t i0) {
  const uint32_t step = blockDim.x * N, H = p.H, first = i0 + threadIdx.x * N;
  Piece<E, N> v[kHold];
#pragma unroll
  for (int c = 0; c < kHold; ++c)
    if (first + c * step < H) {
      const char* from = p.src + t * p.src_stride;
      if (NT)  // the token row has been read before, and is in the cache
        load_piece(v[c], from, start_of<E, N>(first + c * step, H));
      else
        load_once(v[c], from, start_of<E, N>(first + c * step, H));
    }
  for (int j0 = 0; j0 < p.k; j0 += 8) {
    int row[8];
    float w[8];
    rows_of(p, t, j0, row);
    if (WEIGHT) weights_of(p, t, j0, w);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (row[u] < 0) continue;
      char* to = p.dst + (size_t)row[u] * p.dst_stride;
#pragma unroll
      for (int c = 0; c < kHold; ++c)
        if (first + c * step < H)
          store_piece<NT>(WEIGHT ? scaled(v[c], w[u]) : v[c], to,
                          start_of<E, N>(first + c * step, H));
    }
  }
  zero_unnamed<E, N>(p, t, i0, min(i0 + kHold * step, H));
}

template <typename E, int N, bool WEIGHT>
__global__ __launch_bounds__(kThreads) void spread_rows(RowsArgs p) {
  const uint32_t span = kHold * blockDim.x * N;
  for (uint32_t t = blockIdx.x; t < (uint32_t)p.T; t += gridDim.x)
    for (uint32_t i0 = blockIdx.y * span; i0 < (uint32_t)p.H; i0 += gridDim.y * span)
      spread_span<E, N, WEIGHT, false>(p, t, i0);
}

// gather: a thread sums a piece of a token row over its k rows, the loads of eight
// rows in flight.  An absent pick's load goes to row 0 and its sum is skipped, never
// multiplied, so what that row holds does not matter.
template <typename E, int N>
__global__ __launch_bounds__(kThreads) void gather_rows(RowsArgs p) {
  const uint32_t step = blockDim.x * N, H = p.H;
  for (uint32_t t = blockIdx.x; t < (uint32_t)p.T; t += gridDim.x) {
    for (uint32_t i = blockIdx.y * step + threadIdx.x * N; i < H; i += gridDim.y * step) {
      const uint32_t at = start_of<E, N>(i, H);
      float acc[N] = {};
      for (int j0 = 0; j0 < p.k; j0 += 8) {
        int row[8];
        float w[8];
        Piece<E, N> v[8];
        rows_of(p, t, j0, row);
        weights_of(p, t, j0, w);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (j0 + u < p.k) load_once(v[u], p.src + (size_t)max(row[u], 0) * p.src_stride, at);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (row[u] >= 0) {
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] = fmaf(w[u], to_f32<E>(v[u].e[e]), acc[e]);
          }
      }
      Piece<E, N> o;
#pragma unroll
      for (int e = 0; e < N; ++e) o.e[e] = from_f32<E>(acc[e]);
      store_piece<true>(o, p.dst + t * p.dst_stride, at);
    }
  }
}

// Sums of KP values over the workgroup: a wave's by shuffles, then the waves' in
// ascending order through LDS.  Thread j < KP gets value j.
template <int KP>
__device__ __forceinline__ float token_sums(const float (&acc)[KP]) {
  __shared__ float part[kDotThreads / kWave][KP];
  const int wave = threadIdx.x / kWave;
  __syncthreads();  // the sums of the token before have been read
#pragma unroll
  for (int j = 0; j < KP; ++j) {
    const float s = wave_sum_f32(acc[j]);
    if ((threadIdx.x & 63) == j) part[wave][j] = s;
  }
  __syncthreads();
  if (threadIdx.x >= KP) return 0.0f;
  float s = part[0][threadIdx.x];
  for (unsigned v = 1; v < blockDim.x / kWave; ++v) s += part[v][threadIdx.x];
  return s;
}

// The backward calls with the weight's gradient: spread or gather, and the dot
// products of the token's k rows with its token row.  SPREAD: src holds the token
// rows, other the rows (the token row is read again for the spread, from the
// cache); otherwise src holds the rows, other the token rows.
template <typename E, int N, int KP, bool SPREAD>
__global__ __launch_bounds__(kDotThreads) void rows_dot(RowsArgs p) {
  const uint32_t step = blockDim.x * N, H = p.H;
  const char* tokens = SPREAD ? p.src : p.other;
  const char* rows = SPREAD ? p.other : p.src;
  const size_t token_stride = SPREAD ? p.src_stride : p.other_stride;
  const size_t row_stride = SPREAD ? p.other_stride : p.src_stride;
  for (uint32_t t = blockIdx.x; t < (uint32_t)p.T; t += gridDim.x) {
    float dot[KP] = {};
    for (uint32_t i = threadIdx.x * N; i < H; i += step) {
      const uint32_t at = start_of<E, N>(i, H), twice = i - at;  // elements counted before
      Piece<E, N> tok;
      load_piece(tok, tokens + t * token_stride, at);
      float acc[N] = {};
#pragma unroll
      for (int j0 = 0; j0 < KP; j0 += 8) {
        int row[8];
        float w[8];
        Piece<E, N> v[8];
        rows_of(p, t, j0, row);
        weights_of(p, t, j0, w);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (j0 + u < p.k) load_once(v[u], rows + (size_t)max(row[u], 0) * row_stride, at);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (row[u] < 0) continue;
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float x = to_f32<E>(v[u].e[e]);
            const float d = fmaf(x, to_f32<E>(tok.e[e]), dot[j0 + u]);
            dot[j0 + u] = e + 1 == N || e >= (int)twice ? d : dot[j0 + u];
            if (!SPREAD) acc[e] = fmaf(w[u], x, acc[e]);
          }
        }
      }
      if (!SPREAD) {
        Piece<E, N> o;
#pragma unroll
        for (int e = 0; e < N; ++e) o.e[e] = from_f32<E>(acc[e]);
        store_piece<true>(o, p.dst + t * p.dst_stride, at);
      }
    }
    if (SPREAD) {  // apart from the reads, so that each row is written in one stretch
      for (uint32_t i0 = 0; i0 < H; i0 += kHold * step) {
        if (p.weight)
          spread_span<E, N, true, true>(p, t, i0);
        else
          spread_span<E, N, false, true>(p, t, i0);
      }
    }
    const float s = token_sums<KP>(dot);
    if (threadIdx.x < KP && (int)threadIdx.x < p.k)
      p.dweight[(size_t)t * p.k + threadIdx.x] = s;
  }
}

// pos[perm[p]] = p, -1 for assignments that perm does not name.  Up to 4096
// assignments one workgroup builds the array in LDS (4096: 3.0 us against 3.9 of a
// fill and a scatter; 16384: 6.9 against 4.3); larger ones take those two.  Should
// perm name an assignment twice, the larger position stands, whatever the order of
// the threads.
__global__ __launch_bounds__(1024) void positions_lds(const int32_t* __restrict__ perm, int n,
                                                      int32_t* __restrict__ pos,
                                                      int32_t* __restrict__ copy) {
  __shared__ int32_t at[kLdsPositions];
  for (int i = threadIdx.x; i < n; i += 1024) at[i] = -1;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 1024) {
    const int a = perm[i];
    if (copy) copy[i] = a;
    if ((unsigned)a < (unsigned)n) atomicMax(&at[a], i);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 1024) pos[i] = at[i];
}

__global__ __launch_bounds__(256) void positions_fill(int n, int32_t* __restrict__ pos) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    pos[i] = -1;
}

__global__ __launch_bounds__(256) void positions_scatter(const int32_t* __restrict__ perm, int n,
                                                         int32_t* __restrict__ pos,
                                                         int32_t* __restrict__ copy) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int a = perm[i];
    if (copy) copy[i] = a;
    if ((unsigned)a < (unsigned)n) atomicMax(&pos[a], (int)i);
  }
}

unsigned blocks_for(int64_t work, int per) {
  const int64_t b = (work + per - 1) / per;
  return (unsigned)(b < kMaxGrid ? b : kMaxGrid);
}

int shape_status(int T, int k) {
  if (T < 0 || k <= 0) return MOE_EINVAL;
  if (k > MOE_MAX_K || (int64_t)T * k > INT32_MAX) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// Argument checks common to the four calls; src_rows and other_rows say which
// side holds the T*k rows.
int rows_status(const moe_rows_args* a, bool src_rows, bool backward) {
  if (!a) return MOE_EINVAL;
  const int s = shape_status(a->T, a->k);
  if (s != MOE_OK) return s;
  const size_t e = dtype_bytes(a->dtype);
  if (a->H <= 0 || e == 0) return MOE_EINVAL;
  if (a->H > (1 << 30)) return MOE_EUNSUPPORTED;
  if (a->T == 0) return MOE_OK;
  const size_t H = (size_t)a->H;
  if (!a->pos || !a->src || !a->dst) return MOE_EINVAL;
  if (!aligned(a->pos, 4) || !aligned(a->perm, 4) || !aligned(a->weight, 4) ||
      !aligned(a->dweight, 4) || !aligned(a->src, e) || !aligned(a->dst, e) ||
      !aligned(a->other, e))
    return MOE_EINVAL;
  if (a->src_stride < H || a->dst_stride < H) return MOE_EINVAL;
  if (src_rows && a->perm) return MOE_EINVAL;
  if (backward) {
    if ((a->dweight != nullptr) != (a->other != nullptr)) return MOE_EINVAL;
    if (a->dweight && a->other_stride < H) return MOE_EINVAL;
  } else if (a->dweight || a->other) {
    return MOE_EINVAL;
  }
  return MOE_OK;
}

template <typename E, int N, bool SPREAD>
void launch_pieces(const RowsArgs& p, hipStream_t stream) {
  const int pieces = (p.H + N - 1) / N;
  // two pieces a thread and more where a row is only copied, one where it is summed
  const int want = SPREAD && !p.dweight ? pieces / 2 : pieces;
  int threads = kWave;
  while (threads < want && threads < (p.dweight ? kDotThreads : kThreads)) threads *= 2;
  const unsigned grid = blocks_for(p.T, 1);
  if (p.dweight) {
    if (p.k <= 8)
      rows_dot<E, N, 8, SPREAD><<<grid, threads, 0, stream>>>(p);
    else if (p.k <= 16)
      rows_dot<E, N, 16, SPREAD><<<grid, threads, 0, stream>>>(p);
    else
      rows_dot<E, N, 32, SPREAD><<<grid, threads, 0, stream>>>(p);
    return;
  }
  const int per = SPREAD ? threads * kHold : threads, across = (pieces + per - 1) / per;
  const dim3 g(grid, across < 1024 ? across : 1024);
  if (!SPREAD)
    gather_rows<E, N><<<g, threads, 0, stream>>>(p);
  else if (p.weight)
    spread_rows<E, N, true><<<g, threads, 0, stream>>>(p);
  else
    spread_rows<E, N, false><<<g, threads, 0, stream>>>(p);
}

template <typename E, bool SPREAD>
void launch_rows(const RowsArgs& p, hipStream_t stream) {
  if (p.H >= Piece<E>::kN)
    launch_pieces<E, Piece<E>::kN, SPREAD>(p, stream);
  else
    launch_pieces<E, 1, SPREAD>(p, stream);
}

template <bool SPREAD>
int rows_launch(const moe_rows_args* a, hipStream_t stream) {
  if (a->T == 0) return MOE_OK;
  const size_t e = dtype_bytes(a->dtype);
  RowsArgs p{};
  p.T = a->T, p.H = a->H, p.k = a->k, p.n = a->T * a->k;
  p.perm = a->perm, p.pos = a->pos, p.weight = a->weight;
  p.src = (const char*)a->src, p.dst = (char*)a->dst, p.other = (const char*)a->other;
  p.dweight = a->dweight;
  p.src_stride = a->src_stride * e, p.dst_stride = a->dst_stride * e;
  p.other_stride = a->other_stride * e;
  if (a->dtype == MOE_DT_BF16)
    launch_rows<Bf16, SPREAD>(p, stream);
  else if (a->dtype == MOE_DT_FP16)
    launch_rows<Fp16, SPREAD>(p, stream);
  else
    launch_rows<float, SPREAD>(p, stream);
  return hip_status();
}

}  // namespace

extern "C" MOE_EXPORT int moe_positions(const int32_t* perm, int T, int k, int32_t* pos,
                                        int32_t* perm_copy, hipStream_t stream) {
  const int s = shape_status(T, k);
  if (s != MOE_OK) return s;
  if (T == 0) return MOE_OK;
  if (!perm || !pos || !aligned(perm, 4) || !aligned(pos, 4) || !aligned(perm_copy, 4))
    return MOE_EINVAL;
  const int n = T * k;
  if (n <= kLdsPositions) {
    positions_lds<<<1, 1024, 0, stream>>>(perm, n, pos, perm_copy);
  } else {
    positions_fill<<<blocks_for(n, 256), 256, 0, stream>>>(n, pos);
    positions_scatter<<<blocks_for(n, 256), 256, 0, stream>>>(perm, n, pos, perm_copy);
  }
  return hip_status();
}

extern "C" MOE_EXPORT int moe_dispatch(const moe_rows_args* a, hipStream_t stream) {
  const int s = rows_status(a, false, false);
  return s != MOE_OK ? s : rows_launch<true>(a, stream);
}

extern "C" MOE_EXPORT int moe_dispatch_backward(const moe_rows_args* a, hipStream_t stream) {
  const int s = rows_status(a, true, true);
  return s != MOE_OK ? s : rows_launch<false>(a, stream);
}

extern "C" MOE_EXPORT int moe_combine(const moe_rows_args* a, hipStream_t stream) {
  const int s = rows_status(a, true, false);
  return s != MOE_OK ? s : rows_launch<false>(a, stream);
}

extern "C" MOE_EXPORT int moe_combine_backward(const moe_rows_args* a, hipStream_t stream) {
  const int s = rows_status(a, false, true);
  return s != MOE_OK ? s : rows_launch<true>(a, stream);
}
