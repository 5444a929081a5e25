// Log probabilities of given tokens under rows of logits, with the entropy and
// the top alternatives of each row, and their gradient.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/dora.h"
#include "elem.h"
#include "entry.h"
#include "kernels.h"

namespace dora {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kU = 4;   // vectors in flight per thread
// HIP holds the threads of a launch below 2^32: more rows than this share
// workgroups.
constexpr int64_t kMaxGrid = int64_t(1) << 23;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
// Beyond this |lse| the float32 lse itself is too coarse for exp(l - lse) (its
// half ulp is 3e-5 here), and the backward takes the row's maximum and sum anew.
constexpr float kCoarseLse = 1024.f;

// A row is read by up to kMaxSplits workgroups, in chunks of at most kMaxChunk
// elements (their group maxima stay in LDS).
constexpr int64_t kMaxSplits = 128;
constexpr int64_t kMaxChunk = 131072;
constexpr int kMaxTop = DORA_LOGPROB_MAX_TOP;

// Larger of two, NaN if either is (v_maximum3_f32).
__device__ __forceinline__ float maxnan(float a, float b) {
  return __builtin_elementwise_maximum(a, b);
}

// Whole numbers in the order of the floats: NaN above +inf, -0 equal to +0.
__device__ __forceinline__ uint32_t order_bits(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o) {
  return __uint_as_float((o >> 31) ? o & 0x7fffffffu : ~o);
}
// Larger value first, then the lower index.  No key of a logit is 0.
__device__ __forceinline__ uint64_t order_key(float v, uint32_t index) {
  return ((uint64_t)order_bits(v) << 32) | (uint32_t)~index;
}

// Running statistics of a set of logits under a scale: m their maximum,
// s = sum exp2(d), u = sum d exp2(d) with d = (z - m) scale log2(e).  The
// difference is taken before the scaling, so rows of the type's lowest values
// cannot overflow; a logit of -inf adds 0 to both sums; a NaN or +inf makes s NaN.
struct Stat {
  float m, s, u;
};
constexpr float kFloor = -200.f;   // exp2 of this is 0 in float32
__device__ __forceinline__ Stat empty_stat() { return {kNegInf, 0.f, 0.f}; }

__device__ __forceinline__ void rescale(Stat& a, float m, float c2) {
  if (a.m == kNegInf) {   // nothing in it: keep the zeros
    a.m = m;
    return;
  }
  const float d = (a.m - m) * c2;
  const float f = __builtin_amdgcn_exp2f(d);
  a.u = f * fmaf(a.s, fmaxf(d, kFloor), a.u);
  a.s *= f;
  a.m = m;
}
__device__ __forceinline__ Stat merge(Stat a, Stat b, float c2) {
  const float m = maxnan(a.m, b.m);
  rescale(a, m, c2);
  rescale(b, m, c2);
  return {m, a.s + b.s, a.u + b.u};
}

template <int N>
__device__ __forceinline__ void add_logits(Stat& a, const float* v, float c2) {
  float m = v[0];
#pragma unroll
  for (int q = 1; q < N; ++q) m = maxnan(m, v[q]);
  m = maxnan(m, a.m);
  rescale(a, m, c2);
  const float ref = m == kNegInf ? 0.f : m;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const float d = (v[q] - ref) * c2;
    const float e = __builtin_amdgcn_exp2f(d);
    a.s += e;
    a.u = fmaf(e, fmaxf(d, kFloor), a.u);
  }
}

// The workgroup's merged statistics, to every thread; `lds` holds kWaves.
__device__ __forceinline__ Stat block_stat(Stat a, float c2, Stat* lds) {
  float m = a.m;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = maxnan(m, __shfl_xor(m, off, 64));
  rescale(a, m, c2);
  a.s = wave_sum(a.s);
  a.u = wave_sum(a.u);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = a;
  __syncthreads();
  a = lds[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) a = merge(a, lds[w], c2);
  return a;
}

// One row's results from its statistics.
struct RowOut {
  float logp, entropy, lse, ref, log_s;
  bool none;   // nothing left of the row
};
__device__ __forceinline__ RowOut row_out(const Stat& a, float at, float scale) {
  RowOut r;
  r.none = a.m == kNegInf;
  r.ref = r.none ? 0.f : a.m;
  r.log_s = logf(a.s);
  r.logp = r.none ? kNegInf : (at - r.ref) * scale - r.log_s;
  r.entropy = r.none ? 0.f : r.log_s - a.u * kLn2 / a.s;
  r.lse = fmaf(r.ref, scale, r.log_s);
  return r;
}

// ---- top alternatives --------------------------------------------------------------
// While a chunk streams past, the maximum of every group of 4 consecutive
// vectors goes to LDS.  The top k elements lie in the k groups that are first by
// (maximum falling, index rising): an element outside them has k groups before
// its own, each with an element that comes before it.  The same holds one level
// up for runs of consecutive groups, one run per thread.  So three rounds of
// counting ranks suffice, each over few candidates: the k best of 256 runs; the
// k best groups of those runs; the k best elements of those groups, which are
// read again (from cache: 64 bytes each).  A candidate below the k-th of the
// round before is dropped first, which leaves little more than k of them unless
// many are equal.  Nothing depends on the order or distribution of the logits but
// the time, and that only through ties.
constexpr int kListCap = 2048;   // kMaxTop * max(groups per run, elements per group)
struct TopLds {
  uint64_t list[kListCap];
  uint32_t run[kThreads];     // order bits of the runs' maxima
  uint32_t chosen[kMaxTop];   // the runs or groups of the round
  uint32_t count, bound;
};

__device__ __forceinline__ int rank_in(uint64_t key, const uint64_t* list, int n) {
  int r = 0;
#pragma unroll 4
  for (int i = 0; i < n; ++i) r += list[i] > key ? 1 : 0;
  return r;
}

// Keys of the k first elements of row[0, n), in order, to put(rank, key);
// n >= k.  `group` holds the maxima of groups of G elements.
template <bool BF, typename Put>
__device__ void select_top(const typename Elem<BF>::T* row, int64_t n, const float* group, int k,
                           Put put) {
  __shared__ TopLds t;
  constexpr int G = 4 * Elem<BF>::kN;
  const int tid = threadIdx.x;
  const int ng = (int)((n + G - 1) / G);
  const int run = (ng + kThreads - 1) / kThreads;   // groups per run
  const int runs = (ng + run - 1) / run;
  // runs
  const int g0 = tid * run, g1 = min(ng, g0 + run);
  uint32_t best = 0;
  for (int g = g0; g < g1; ++g) best = max(best, order_bits(group[g]));
  t.run[tid] = best;
  if (tid == 0) {
    t.count = 0;
    t.bound = 0;
  }
  __syncthreads();
  int r = 0;
#pragma unroll 4
  for (int i = 0; i < kThreads; i += 4) {
    const u32x4 o = *reinterpret_cast<const u32x4*>(&t.run[i]);
#pragma unroll
    for (int q = 0; q < 4; ++q) r += (o[q] > best || (o[q] == best && i + q < tid)) ? 1 : 0;
  }
  const bool in = tid < runs && r < k;
  if (in && r == k - 1) t.bound = best;
  __syncthreads();
  // groups of the chosen runs
  const uint32_t bound = t.bound;
  if (in) {
    for (int g = g0; g < g1; ++g) {
      const uint32_t o = order_bits(group[g]);
      if (o >= bound) t.list[atomicAdd(&t.count, 1u)] = ((uint64_t)o << 32) | (uint32_t)~(uint32_t)g;
    }
  }
  __syncthreads();
  int m = (int)t.count;
  for (int i = tid; i < m; i += kThreads) {
    const uint64_t key = t.list[i];
    const int rank = rank_in(key, t.list, m);
    if (rank < k) t.chosen[rank] = ~(uint32_t)key;
    if (rank == k - 1) t.bound = (uint32_t)(key >> 32);
  }
  const int picked = min(m, k);
  __syncthreads();
  // elements of the chosen groups
  const uint32_t least = m >= k ? t.bound : 0u;
  if (tid == 0) t.count = 0;
  __syncthreads();
  for (int i = tid; i < picked * G; i += kThreads) {
    const int64_t j = (int64_t)t.chosen[i / G] * G + i % G;
    if (j < n) {
      const uint64_t key = order_key(Elem<BF>::get(row + j), (uint32_t)j);
      if ((uint32_t)(key >> 32) >= least) t.list[atomicAdd(&t.count, 1u)] = key;
    }
  }
  __syncthreads();
  m = (int)t.count;
  for (int i = tid; i < m; i += kThreads) {
    const uint64_t key = t.list[i];
    const int rank = rank_in(key, t.list, m);
    if (rank < k) put(rank, key);
  }
}

// Chunk blockIdx.x of a row (or, with one chunk, the whole row and its results).
// Loads are kU vectors ahead of the arithmetic; per element the loop costs a
// subtraction, two products, an exponential, a maximum and two sums.
template <bool BF, bool TOP, bool SPLIT>
__global__ __launch_bounds__(kThreads) void dora_logprob_fwd(
    const void* logits, int64_t ld, const int64_t* targets, float* logp, float* entropy, float* lse,
    float* top_logp, int64_t* top_index, Stat* part, uint64_t* part_top, int64_t rows, int64_t V,
    int64_t chunk, int top, float scale) {
  using E = Elem<BF>;
  using T = typename E::T;
  constexpr int kStep = kThreads * E::kN;
  extern __shared__ float group[];
  __shared__ Stat lds[kWaves];
  const float c2 = scale * kLog2e;
  const int64_t lo = (int64_t)blockIdx.x * chunk;
  const int64_t n = min(V - lo, chunk);
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const int64_t y = targets[row];
    if (y < 0 || y >= V) {
      if (SPLIT) continue;   // the join writes its zeros
      if (threadIdx.x == 0) {
        logp[row] = 0.f;
        if (entropy) entropy[row] = 0.f;
        if (lse) lse[row] = 0.f;
      }
      if (TOP && (int)threadIdx.x < top) {
        top_logp[row * top + threadIdx.x] = 0.f;
        top_index[row * top + threadIdx.x] = -1;
      }
      continue;
    }
    const T* z = reinterpret_cast<const T*>(logits) + row * ld;
    const float at = SPLIT ? 0.f : E::get(z + y);
    z += lo;
    Stat a = empty_stat();
    auto group_max = [&](const float* v, int64_t j) {
      float m = v[0];
#pragma unroll
      for (int q = 1; q < E::kN; ++q) m = maxnan(m, v[q]);
      m = maxnan(m, __shfl_xor(m, 1, 64));
      m = maxnan(m, __shfl_xor(m, 2, 64));
      if ((threadIdx.x & 3) == 0 && j < n) group[j / (4 * E::kN)] = m;
    };
    int64_t j = (int64_t)threadIdx.x * E::kN;
    int64_t left = n;
    for (; left >= kStep * kU; left -= kStep * kU, j += kStep * kU) {
      float v[kU][E::kN];
#pragma unroll
      for (int u = 0; u < kU; ++u) E::load(z + j + u * kStep, v[u]);
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (TOP) group_max(v[u], j + u * kStep);
      add_logits<kU * E::kN>(a, &v[0][0], c2);
    }
    for (; left > 0; left -= kStep, j += kStep) {
      float v[E::kN];
      load_part<BF>(z, j, n, kNegInf, v);
      if (TOP) group_max(v, j);
      add_logits<E::kN>(a, v, c2);
    }
    a = block_stat(a, c2, lds);   // its barrier also completes the group maxima
    RowOut out;
    if (SPLIT) {
      if (threadIdx.x == 0) part[row * gridDim.x + blockIdx.x] = a;
    } else {
      out = row_out(a, at, scale);
      if (threadIdx.x == 0) {
        logp[row] = out.logp;
        if (entropy) entropy[row] = out.entropy;
        if (lse) lse[row] = out.lse;
      }
    }
    if constexpr (TOP) {
      const int k = (int)min((int64_t)top, n);
      uint64_t* mine = SPLIT ? part_top + (row * gridDim.x + blockIdx.x) * top : nullptr;
      if (SPLIT && k < top && (int)threadIdx.x >= k && (int)threadIdx.x < top)
        mine[threadIdx.x] = 0;   // a chunk shorter than the list
      select_top<BF>(z, n, group, k, [&](int rank, uint64_t key) {
        const uint32_t index = ~(uint32_t)key;
        if (SPLIT) {
          mine[rank] = (key & 0xffffffff00000000ull) | (uint32_t)~(index + (uint32_t)lo);
        } else {
          const float v = order_value((uint32_t)(key >> 32));
          top_index[row * top + rank] = index;
          top_logp[row * top + rank] = out.none ? kNegInf : (v - out.ref) * scale - out.log_s;
        }
      });
    }
    __syncthreads();   // LDS is written again for the next row
  }
}

// Joins the chunks of a row: their statistics in order, and the first k of their
// sorted lists.  A key below the k-th best of the lists' heads (where there are k
// lists) or below any list's last is out; at most kMaxTop^2 remain.
constexpr int kJoinCap = kMaxTop * kMaxTop;
template <bool BF, bool TOP>
__global__ __launch_bounds__(kThreads) void dora_logprob_join(
    const void* logits, int64_t ld, const int64_t* targets, const Stat* part,
    const uint64_t* part_top, int splits, float* logp, float* entropy, float* lse, float* top_logp,
    int64_t* top_index, int64_t rows, int64_t V, int top, float scale) {
  using E = Elem<BF>;
  __shared__ Stat stats[kMaxSplits];
  __shared__ uint64_t heads[TOP ? kMaxSplits : 1];
  __shared__ uint64_t list[TOP ? kJoinCap : 1];
  __shared__ uint32_t count;
  __shared__ unsigned long long bound;
  const int tid = threadIdx.x;
  const float c2 = scale * kLog2e;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t y = targets[row];
    if (y < 0 || y >= V) {
      if (tid == 0) {
        logp[row] = 0.f;
        if (entropy) entropy[row] = 0.f;
        if (lse) lse[row] = 0.f;
      }
      if (TOP && tid < top) {
        top_logp[row * top + tid] = 0.f;
        top_index[row * top + tid] = -1;
      }
      continue;
    }
    const float at = E::get(reinterpret_cast<const typename E::T*>(logits) + row * ld + y);
    const uint64_t* lists = TOP ? part_top + row * splits * top : nullptr;
    if (tid < splits) {
      stats[tid] = part[row * splits + tid];
      if (TOP) heads[tid] = lists[(int64_t)tid * top];
    }
    if (tid == 0) {
      count = 0;
      bound = 0;
    }
    __syncthreads();
    Stat a = stats[0];
    for (int i = 1; i < splits; ++i) a = merge(a, stats[i], c2);
    const RowOut out = row_out(a, at, scale);
    if (tid == 0) {
      logp[row] = out.logp;
      if (entropy) entropy[row] = out.entropy;
      if (lse) lse[row] = out.lse;
    }
    if (TOP) {
      if (tid < splits) {
        const uint64_t last = lists[(int64_t)tid * top + top - 1];
        atomicMax(&bound, (unsigned long long)last);
        if (splits >= top && rank_in(heads[tid], heads, splits) == top - 1)
          atomicMax(&bound, (unsigned long long)heads[tid]);
      }
      __syncthreads();
      const uint64_t least = max((uint64_t)bound, (uint64_t)1);   // 0 pads short lists
      for (int i = tid; i < splits * top; i += kThreads) {
        const uint64_t key = lists[i];
        if (key >= least) list[atomicAdd(&count, 1u)] = key;
      }
      __syncthreads();
      const int m = (int)count;
      for (int i = tid; i < m; i += kThreads) {
        const uint64_t key = list[i];
        const int rank = rank_in(key, list, m);
        if (rank < top) {
          const float v = order_value((uint32_t)(key >> 32));
          top_index[row * top + rank] = (uint32_t)~(uint32_t)key;
          top_logp[row * top + rank] = out.none ? kNegInf : (v - out.ref) * scale - out.log_s;
        }
      }
    }
    __syncthreads();
  }
}

template <bool BF>
__global__ __launch_bounds__(kThreads) void dora_logprob_bwd(
    const float* g_logp, const float* g_entropy, const void* logits, int64_t ld,
    const int64_t* targets, const float* lse, const float* entropy, void* grad, int64_t rows,
    int64_t V, float scale) {
  using E = Elem<BF>;
  using T = typename E::T;
  __shared__ Stat lds[kWaves];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
  __syncthreads();   // the previous row's reductions have been read
  const T* z = reinterpret_cast<const T*>(logits) + row * ld;
  T* gz = reinterpret_cast<T*>(grad) + row * V;
  const int64_t y = targets[row];
  bool zero = y < 0 || y >= V;
  float ref = 0.f, log_s = 0.f;
  if (!zero) {
    log_s = lse[row];
    if (!(fabsf(log_s) <= kCoarseLse)) {
      Stat st = empty_stat();
      for (int64_t j = (int64_t)threadIdx.x * E::kN; j < V; j += kThreads * E::kN) {
        float v[E::kN];
        load_part<BF>(z, j, V, kNegInf, v);
        add_logits<E::kN>(st, v, scale * kLog2e);
      }
      const RowOut r = row_out(block_stat(st, scale * kLog2e, lds), 0.f, scale);
      zero = r.none;
      ref = r.ref;
      log_s = r.log_s;
    }
  }
  const float a = g_logp ? g_logp[row] : 0.f;
  const float b = g_entropy ? g_entropy[row] : 0.f;
  const float H = g_entropy ? entropy[row] : 0.f;
  for (int64_t j = (int64_t)threadIdx.x * E::kN; j < V; j += kThreads * E::kN) {
    float v[E::kN], o[E::kN];
    load_part<BF>(z, j, V, kNegInf, v);
#pragma unroll
    for (int q = 0; q < E::kN; ++q) {
      const float d = fmaf(v[q] - ref, scale, -log_s);
      const float p = exp2f(d * kLog2e);
      const float inner = p > 0.f ? d + H : 0.f;
      float g = -p * fmaf(b, inner, a);
      if (j + q == y) g += a;
      o[q] = zero ? 0.f : g * scale;
    }
    store_part<BF>(gz, j, V, o);
  }
  }
}

constexpr int64_t kLimit = int64_t(1) << 31;
constexpr int64_t kMaxVocab = kMaxSplits * kMaxChunk;   // 2^24

bool shape_ok(const dora_logprob_shape& s) {
  return s.rows >= 0 && s.rows < kLimit && s.vocab >= 1 && s.vocab <= kMaxVocab && s.ld >= s.vocab &&
         s.ld < kLimit && s.top >= 0 && s.top <= DORA_LOGPROB_MAX_TOP && s.top <= s.vocab;
}
bool dtype_ok(const dora_logprob_shape& s) { return s.dtype == DORA_F32 || s.dtype == DORA_BF16; }

int check_shape(const dora_logprob_shape* s) {
  if (!s) return DORA_ERR_NULL;
  if (s->reserved != 0 || !std::isfinite(s->scale) || s->scale <= 0.f) return DORA_ERR_FLAGS;
  if (!dtype_ok(*s)) return DORA_ERR_DTYPE;
  if (!shape_ok(*s)) return DORA_ERR_SHAPE;
  return DORA_OK;
}

// How many workgroups read a row.  With rows enough to give every CU a few
// workgroups each row is one workgroup's; below that rows are cut until about
// kWantBlocks workgroups run, no chunk under kMinChunk elements.
constexpr int64_t kWantBlocks = 1024;
constexpr int64_t kMinChunk = 4096;
struct Plan {
  int64_t chunk, splits;
  size_t stat_bytes, top_bytes;
};
Plan plan(const dora_logprob_shape& s) {
  Plan p;
  const int64_t most = std::min(kMaxSplits, std::max<int64_t>(1, s.vocab / kMinChunk));
  const int64_t want = std::max<int64_t>(1, kWantBlocks / std::max<int64_t>(1, s.rows));
  const int64_t least = (s.vocab + kMaxChunk - 1) / kMaxChunk;
  const int64_t n = std::max(least, std::min(want, most));
  p.chunk = std::min(kMaxChunk, ((s.vocab + n - 1) / n + 2047) / 2048 * 2048);
  p.splits = (s.vocab + p.chunk - 1) / p.chunk;
  const int64_t parts = p.splits > 1 ? s.rows * p.splits : 0;
  p.stat_bytes = (size_t)((parts * (int64_t)sizeof(Stat) + 15) / 16 * 16);
  p.top_bytes = (size_t)(parts * s.top * 8);
  return p;
}

template <bool BF, bool TOP, bool SPLIT>
hipError_t launch_fwd(const dora_logprob_shape& s, const Plan& p, const void* logits,
                      const int64_t* targets, float* logp, float* entropy, float* lse,
                      float* top_logp, int64_t* top_index, Stat* part, uint64_t* part_top,
                      hipStream_t st) {
  const unsigned rows = (unsigned)std::min<int64_t>(s.rows, 65535);
  const size_t groups = TOP ? (size_t)(std::min(p.chunk, s.vocab) + 4 * Elem<BF>::kN - 1) /
                                  (4 * Elem<BF>::kN) * sizeof(float)
                            : 0;
  {
    LaunchTimer t("logprob_fwd", st);
    hipLaunchKernelGGL((dora_logprob_fwd<BF, TOP, SPLIT>), dim3((unsigned)p.splits, rows),
                       dim3(kThreads), groups, st, logits, s.ld, targets, logp, entropy, lse,
                       top_logp, top_index, part, part_top, s.rows, s.vocab, p.chunk, (int)s.top,
                       s.scale);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (!SPLIT) return hipSuccess;
  LaunchTimer t("logprob_join", st);
  hipLaunchKernelGGL((dora_logprob_join<BF, TOP>), dim3((unsigned)std::min(s.rows, kMaxGrid)),
                     dim3(kThreads), 0, st, logits, s.ld, targets, part, part_top, (int)p.splits,
                     logp, entropy, lse, top_logp, top_index, s.rows, s.vocab, (int)s.top, s.scale);
  return hipGetLastError();
}

template <bool BF>
hipError_t forward(const dora_logprob_shape& s, const void* logits, const int64_t* targets,
                   float* logp, float* entropy, float* lse, float* top_logp, int64_t* top_index,
                   void* ws, hipStream_t st) {
  const Plan p = plan(s);
  Stat* part = reinterpret_cast<Stat*>(ws);
  uint64_t* part_top =
      ws ? reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(ws) + p.stat_bytes) : nullptr;
  auto go = [&](auto fn) {
    return fn(s, p, logits, targets, logp, entropy, lse, top_logp, top_index, part, part_top, st);
  };
  if (p.splits > 1)
    return s.top > 0 ? go(launch_fwd<BF, true, true>) : go(launch_fwd<BF, false, true>);
  return s.top > 0 ? go(launch_fwd<BF, true, false>) : go(launch_fwd<BF, false, false>);
}

template <bool BF>
hipError_t backward(const dora_logprob_shape& s, const float* g_logp, const float* g_entropy,
                    const void* logits, const int64_t* targets, const float* lse,
                    const float* entropy, void* grad, hipStream_t st) {
  LaunchTimer t("logprob_bwd", st);
  hipLaunchKernelGGL((dora_logprob_bwd<BF>), dim3((unsigned)std::min(s.rows, kMaxGrid)), dim3(kThreads),
                     0, st, g_logp, g_entropy, logits, s.ld, targets, lse, entropy, grad, s.rows, s.vocab, s.scale);
  return hipGetLastError();
}

}  // namespace
}  // namespace dora

using namespace dora;

extern "C" {

DORA_API size_t dora_token_logprob_workspace_bytes(const dora_logprob_shape* shape) {
  if (!shape || !dtype_ok(*shape) || !shape_ok(*shape)) return 0;
  const Plan p = plan(*shape);
  return p.stat_bytes + p.top_bytes;
}

DORA_API int dora_token_logprob_forward(const dora_logprob_shape* shape, const void* logits,
                                        const int64_t* targets, float* logp, float* entropy,
                                        float* lse, float* top_logp, int64_t* top_index, void* ws,
                                        size_t ws_bytes, void* hip_stream) {
  DORA_CHECK(check_shape(shape));
  const dora_logprob_shape& s = *shape;
  const size_t e = s.dtype == DORA_BF16 ? 2 : 4;
  const bool empty = s.rows == 0;
  DORA_CHECK(check_elem(logits, e, empty));
  DORA_CHECK(check_elem(targets, 8, empty));
  DORA_CHECK(check_elem(logp, 4, empty));
  DORA_CHECK(check_elem(entropy, 4, true));
  DORA_CHECK(check_elem(lse, 4, true));
  DORA_CHECK(check_elem(top_logp, 4, empty || s.top == 0));
  DORA_CHECK(check_elem(top_index, 8, empty || s.top == 0));
  DORA_CHECK(check_ws(ws, ws_bytes, dora_token_logprob_workspace_bytes(shape)));
  if (empty) return DORA_OK;
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  HIP_TRY(s.dtype == DORA_BF16
              ? forward<true>(s, logits, targets, logp, entropy, lse, top_logp, top_index, ws, st)
              : forward<false>(s, logits, targets, logp, entropy, lse, top_logp, top_index, ws, st));
  return DORA_OK;
}

DORA_API int dora_token_logprob_backward(const dora_logprob_shape* shape, const float* grad_logp,
                                         const float* grad_entropy, const void* logits,
                                         const int64_t* targets, const float* lse,
                                         const float* entropy, void* grad_logits,
                                         void* hip_stream) {
  DORA_CHECK(check_shape(shape));
  const dora_logprob_shape& s = *shape;
  const size_t e = s.dtype == DORA_BF16 ? 2 : 4;
  const bool empty = s.rows == 0;
  DORA_CHECK(check_elem(grad_logp, 4, true));
  DORA_CHECK(check_elem(grad_entropy, 4, true));
  DORA_CHECK(check_elem(logits, e, empty));
  DORA_CHECK(check_elem(targets, 8, empty));
  DORA_CHECK(check_elem(lse, 4, empty));
  DORA_CHECK(check_elem(entropy, 4, empty || !grad_entropy));
  DORA_CHECK(check_elem(grad_logits, e, empty));
  if (empty) return DORA_OK;
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  HIP_TRY(s.dtype == DORA_BF16
              ? backward<true>(s, grad_logp, grad_entropy, logits, targets, lse, entropy,
                               grad_logits, st)
              : backward<false>(s, grad_logp, grad_entropy, logits, targets, lse, entropy,
                                grad_logits, st));
  return DORA_OK;
}

}  // extern "C"
