// Token rows in the order of the slots and back, with weights and gradients:
// moe_positions, moe_dispatch, moe_dispatch_backward, moe_combine,
// moe_combine_backward.
//
// With a = t*k + j the assignments and pos[a] the row that holds assignment a:
//   spread   row[pos[a]] = w[a] * token[t]                (dispatch; combine's backward)
//   gather   token[t]    = sum_j w[t,j] * row[pos[t,j]]   (combine; dispatch's backward)
// and the weight's gradient is the dot product of the row with the token row
// on the other side.  So two kernel forms serve all four calls.  All of them
// are token-major: a token row is read or written once while its k rows pass,
// where a row-major walk would read each token row k times, from rows far
// apart.  Sums run over ascending j in float32 in one thread, dot products in
// a fixed tree: no atomics, the same result on every call.
#include "elements.hpp"

using namespace moe;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxGrid = 1 << 22;      // workgroups of a launch; they stride over the rest
constexpr int kLdsPositions = 16384;   // assignments that one workgroup orders in LDS

struct RowsArgs {
  int T, H, k, n;          // n = T*k rows
  int lanes;               // threads of a token (a power of two, <= kThreads)
  const int32_t* perm;
  const int32_t* pos;
  const float* weight;
  const void* src;
  void* dst;
  const void* other;
  float* dweight;
  size_t src_stride, dst_stride, other_stride;
};

// The rows of picks j0 .. j0 + 7 of token t: -1 past k and for absent ones.
__device__ __forceinline__ void rows_of(const RowsArgs& p, int t, int j0, int (&row)[8]) {
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    int r = -1;
    if (j0 + u < p.k) r = p.pos[(size_t)t * p.k + j0 + u];
    row[u] = (unsigned)r < (unsigned)p.n ? r : -1;
  }
}

__device__ __forceinline__ void weights_of(const RowsArgs& p, int t, int j0, float (&w)[8]) {
#pragma unroll
  for (int u = 0; u < 8; ++u)
    w[u] = p.weight && j0 + u < p.k ? p.weight[(size_t)t * p.k + j0 + u] : 1.0f;
}

// Row p of the output where perm names no assignment: picks with no slot have
// no row of their own, so these are the last rows, and they are set to zero
// (each by the token whose assignments have the same numbers).
template <typename E>
__device__ __forceinline__ void zero_unnamed(const RowsArgs& p, int t, int i, int left) {
  if (!p.perm) return;
  const Piece<E> zero{};
  for (int j = 0; j < p.k; ++j) {
    const size_t r = (size_t)t * p.k + j;
    if ((unsigned)p.perm[r] >= (unsigned)p.n)
      zero.store_upto((E*)p.dst + r * p.dst_stride + i, left);
  }
}

template <typename E>
__device__ __forceinline__ Piece<E> scaled(const Piece<E>& v, float w) {
  Piece<E> o;
#pragma unroll
  for (int i = 0; i < Piece<E>::kN; ++i) o.e[i] = from_f32<E>(w * to_f32<E>(v.e[i]));
  return o;
}

// spread: every thread reads a 16-byte piece of a token row and stores it k
// times.  Bound by the stores.
template <typename E>
__global__ __launch_bounds__(kThreads) void spread_rows(RowsArgs p) {
  constexpr int N = Piece<E>::kN;
  const int per = kThreads / p.lanes;
  const int lane = threadIdx.x & (p.lanes - 1);
  for (int64_t t0 = (int64_t)blockIdx.x * per + threadIdx.x / p.lanes; t0 < p.T;
       t0 += (int64_t)gridDim.x * per) {
    const int t = (int)t0;
    for (int i = (blockIdx.y * p.lanes + lane) * N; i < p.H; i += gridDim.y * p.lanes * N) {
      const int left = p.H - i;
      Piece<E> v;
      v.load_upto((const E*)p.src + t * p.src_stride + i, left);
      for (int j0 = 0; j0 < p.k; j0 += 8) {
        int row[8];
        float w[8];
        rows_of(p, t, j0, row);
        weights_of(p, t, j0, w);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (row[u] >= 0) {
            const Piece<E> o = p.weight ? scaled<E>(v, w[u]) : v;
            o.store_upto((E*)p.dst + (size_t)row[u] * p.dst_stride + i, left);
          }
      }
      zero_unnamed<E>(p, t, i, left);
    }
  }
}

// gather: every thread sums a 16-byte piece of a token row over its k rows,
// eight loads in flight.  An absent pick's load goes to row 0 and is dropped
// by a select, never multiplied, so what that row holds does not matter.
template <typename E>
__global__ __launch_bounds__(kThreads) void gather_rows(RowsArgs p) {
  constexpr int N = Piece<E>::kN;
  const int per = kThreads / p.lanes;
  const int lane = threadIdx.x & (p.lanes - 1);
  for (int64_t t0 = (int64_t)blockIdx.x * per + threadIdx.x / p.lanes; t0 < p.T;
       t0 += (int64_t)gridDim.x * per) {
    const int t = (int)t0;
    for (int i = (blockIdx.y * p.lanes + lane) * N; i < p.H; i += gridDim.y * p.lanes * N) {
      const int left = p.H - i;
      float acc[N] = {};
      for (int j0 = 0; j0 < p.k; j0 += 8) {
        int row[8];
        float w[8];
        Piece<E> v[8];
        rows_of(p, t, j0, row);
        weights_of(p, t, j0, w);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (j0 + u < p.k)
            v[u].load_upto((const E*)p.src + (size_t)max(row[u], 0) * p.src_stride + i, left);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (row[u] >= 0) {
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] = fmaf(w[u], to_f32<E>(v[u].e[e]), acc[e]);
          }
      }
      Piece<E> o;
#pragma unroll
      for (int e = 0; e < N; ++e) o.e[e] = from_f32<E>(acc[e]);
      o.store_upto((E*)p.dst + t * p.dst_stride + i, left);
    }
  }
}

// Sums of KP values over the threads of a token (64, one wave, or all 256): a
// wave's by shuffles, then the waves' in ascending order through LDS.  Thread
// `lane` < KP of the token gets value `lane`.
template <int KP>
__device__ __forceinline__ float token_sums(const float (&acc)[KP], int lanes, int lane) {
  __shared__ float part[kThreads / kWave][KP];
  const int wave = threadIdx.x / kWave;
  __syncthreads();  // the sums of the token before have been read
#pragma unroll
  for (int j = 0; j < KP; ++j) {
    const float s = wave_sum_f32(acc[j]);
    if ((threadIdx.x & 63) == j) part[wave][j] = s;
  }
  __syncthreads();
  if (lane >= KP) return 0.0f;
  if (lanes == kWave) return part[wave][lane];
  float s = part[0][lane];
#pragma unroll
  for (int v = 1; v < kThreads / kWave; ++v) s += part[v][lane];
  return s;
}

// The backward calls with the weight's gradient: spread or gather, and the dot
// products of the token's k rows with its token row on the way, so neither is
// read twice.  SPREAD: src holds the token rows, other the rows; otherwise src
// holds the rows, other the token rows.  Every workgroup makes the same number
// of rounds for all its tokens, so its barriers are reached by every wave.
template <typename E, int KP, bool SPREAD>
__global__ __launch_bounds__(kThreads) void rows_dot(RowsArgs p) {
  constexpr int N = Piece<E>::kN;
  const int per = kThreads / p.lanes;
  const int lane = threadIdx.x & (p.lanes - 1);
  for (int64_t b = (int64_t)blockIdx.x * per; b < p.T; b += (int64_t)gridDim.x * per) {
    const int64_t t0 = b + threadIdx.x / p.lanes;
    const int t = (int)(t0 < p.T ? t0 : p.T - 1);
    float dot[KP] = {};
    if (t0 < p.T) {
      for (int i = lane * N; i < p.H; i += p.lanes * N) {
        const int left = p.H - i;
        Piece<E> tok;
        if (SPREAD)
          tok.load_upto((const E*)p.src + t * p.src_stride + i, left);
        else
          tok.load_upto((const E*)p.other + t * p.other_stride + i, left);
        float acc[N] = {};
#pragma unroll
        for (int j0 = 0; j0 < KP; j0 += 8) {
          int row[8];
          float w[8];
          Piece<E> v[8];
          rows_of(p, t, j0, row);
          weights_of(p, t, j0, w);
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (j0 + u < p.k) {
              const E* base = SPREAD ? (const E*)p.other + (size_t)max(row[u], 0) * p.other_stride
                                     : (const E*)p.src + (size_t)max(row[u], 0) * p.src_stride;
              v[u].load_upto(base + i, left);
            }
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (row[u] >= 0) {
#pragma unroll
              for (int e = 0; e < N; ++e) {
                const float x = to_f32<E>(v[u].e[e]);
                dot[j0 + u] = fmaf(x, to_f32<E>(tok.e[e]), dot[j0 + u]);
                if (!SPREAD) acc[e] = fmaf(w[u], x, acc[e]);
              }
              if (SPREAD) {
                const Piece<E> o = p.weight ? scaled<E>(tok, w[u]) : tok;
                o.store_upto((E*)p.dst + (size_t)row[u] * p.dst_stride + i, left);
              }
            }
        }
        if (SPREAD) {
          zero_unnamed<E>(p, t, i, left);
        } else {
          Piece<E> o;
#pragma unroll
          for (int e = 0; e < N; ++e) o.e[e] = from_f32<E>(acc[e]);
          o.store_upto((E*)p.dst + t * p.dst_stride + i, left);
        }
      }
    }
    const float s = token_sums<KP>(dot, p.lanes, lane);
    if (t0 < p.T && lane < p.k && lane < KP) p.dweight[(size_t)t * p.k + lane] = s;
  }
}

// pos[perm[p]] = p, -1 for assignments that perm does not name.  Up to 16384
// assignments one workgroup builds the array in LDS; larger ones take a fill
// and a scatter.  Should perm name an assignment twice, the larger position
// stands, whatever the order of the threads.
__global__ __launch_bounds__(1024) void positions_lds(const int32_t* __restrict__ perm, int n,
                                                      int32_t* __restrict__ pos) {
  __shared__ int32_t at[kLdsPositions];
  for (int i = threadIdx.x; i < n; i += 1024) at[i] = -1;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 1024) {
    const int a = perm[i];
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
                                                         int32_t* __restrict__ pos) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int a = perm[i];
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

template <typename E, int KP, bool SPREAD>
void launch_dot(RowsArgs p, hipStream_t stream) {
  const int pieces = (p.H + Piece<E>::kN - 1) / Piece<E>::kN;
  p.lanes = pieces <= 2 * kWave ? kWave : kThreads;
  rows_dot<E, KP, SPREAD><<<blocks_for(p.T, kThreads / p.lanes), kThreads, 0, stream>>>(p);
}

template <typename E, bool SPREAD>
void launch_rows(RowsArgs p, hipStream_t stream) {
  if (p.dweight) {
    if (p.k <= 8)
      launch_dot<E, 8, SPREAD>(p, stream);
    else if (p.k <= 16)
      launch_dot<E, 16, SPREAD>(p, stream);
    else
      launch_dot<E, 32, SPREAD>(p, stream);
    return;
  }
  const int pieces = (p.H + Piece<E>::kN - 1) / Piece<E>::kN;
  p.lanes = 1;
  while (p.lanes < kThreads && p.lanes < pieces) p.lanes *= 2;
  const int across = (pieces + p.lanes - 1) / p.lanes;
  const dim3 grid(blocks_for(p.T, kThreads / p.lanes), across < 1024 ? across : 1024);
  if (SPREAD)
    spread_rows<E><<<grid, kThreads, 0, stream>>>(p);
  else
    gather_rows<E><<<grid, kThreads, 0, stream>>>(p);
}

template <bool SPREAD>
int rows_launch(const moe_rows_args* a, hipStream_t stream) {
  if (a->T == 0) return MOE_OK;
  RowsArgs p{};
  p.T = a->T, p.H = a->H, p.k = a->k, p.n = a->T * a->k;
  p.perm = a->perm, p.pos = a->pos, p.weight = a->weight;
  p.src = a->src, p.dst = a->dst, p.other = a->other, p.dweight = a->dweight;
  p.src_stride = a->src_stride, p.dst_stride = a->dst_stride, p.other_stride = a->other_stride;
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
                                        hipStream_t stream) {
  const int s = shape_status(T, k);
  if (s != MOE_OK) return s;
  if (T == 0) return MOE_OK;
  if (!perm || !pos || !aligned(perm, 4) || !aligned(pos, 4)) return MOE_EINVAL;
  const int n = T * k;
  if (n <= kLdsPositions) {
    positions_lds<<<1, 1024, 0, stream>>>(perm, n, pos);
  } else {
    positions_fill<<<blocks_for(n, 256), 256, 0, stream>>>(n, pos);
    positions_scatter<<<blocks_for(n, 256), 256, 0, stream>>>(perm, n, pos);
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
