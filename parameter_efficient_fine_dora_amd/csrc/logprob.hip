// Log probabilities of given tokens under rows of logits, with the entropy and
// the top alternatives of each row, and their gradient.  With m the row's maximum,
// d_j = scale (z_j - m), s = sum exp(d_j) and u = sum d_j exp(d_j):
//   logp = d_y - log s,  entropy H = log s - u / s,  lse = scale m + log s
//   grad z_j = scale (a ([j = y] - p_j) - b p_j (log p_j + H)), p_j = exp(d_j) / s
// for gradients a of logp and b of entropy.  Statistics are float32, with the
// hardware's exponential (1 ulp) of a difference times the rounded scale log2(e): over
// 4096 rows of 131072 the results are 1.2e-7 off float64's, those of a plain float32
// form 6e-8.  Memory bounds long calls: the forward reads the logits once (4096 x 131072 bf16, an eighth of the rows
// skipped: 146 us, 6.4 TB/s), the gradient reads and writes them once (317 us, 6.3
// TB/s).  Few rows are bound by latency: one of 131072
// bf16 with its top 20 takes 7 us and 4 us for the join.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/dora_finetune.h"
#include "checks.h"
#include "elem.h"
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
constexpr int64_t kMaxSplits = 64;
constexpr int64_t kMaxChunk = 131072;
constexpr int kMaxTop = DORA_LOGPROB_MAX_TOP;

// Larger of two, NaN if either is (v_maximum3_f32).
__device__ __forceinline__ float maxnan(float a, float b) {
  return __builtin_elementwise_maximum(a, b);
}

__device__ __forceinline__ float wave_maxnan(float v) {
  v = maxnan(v, dpp_move<0xB1>(v));
  v = maxnan(v, dpp_move<0x4E>(v));
  v = maxnan(v, dpp_move<0x141>(v));
  v = maxnan(v, dpp_move<0x140>(v));
  return maxnan(maxnan(lane_value(v, 0), lane_value(v, 16)),
                maxnan(lane_value(v, 32), lane_value(v, 48)));
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, __float_as_uint(dpp_move<0xB1>(__uint_as_float(v))));
  v = max(v, __float_as_uint(dpp_move<0x4E>(__uint_as_float(v))));
  v = max(v, __float_as_uint(dpp_move<0x141>(__uint_as_float(v))));
  v = max(v, __float_as_uint(dpp_move<0x140>(__uint_as_float(v))));
  auto at = [&](int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); };
  return max(max(at(0), at(16)), max(at(32), at(48)));
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

// A wave's merged statistics, to every lane.
__device__ __forceinline__ Stat wave_stat(Stat a, float c2) {
  rescale(a, wave_maxnan(a.m), c2);
  a.s = wave_sum(a.s);
  a.u = wave_sum(a.u);
  return a;
}
// A workgroup's, to every thread; `lds` holds WAVES.
template <int WAVES>
__device__ __forceinline__ Stat block_stat(Stat a, float c2, Stat* lds) {
  a = wave_stat(a, c2);
  if (WAVES == 1) return a;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = a;
  __syncthreads();
  float m = lds[0].m;
#pragma unroll
  for (int w = 1; w < WAVES; ++w) m = maxnan(m, lds[w].m);
  Stat sum = {m, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    Stat b = lds[w];
    rescale(b, m, c2);
    sum.s += b.s;
    sum.u += b.u;
  }
  return sum;
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
// up for runs of consecutive groups, one run per thread.  So: the k best runs, by
// bisection over their maxima; the k best groups of those runs and the k best
// elements of those groups, by counting ranks among the few that are not below
// the k-th of the step before.  The groups' elements are read again (from cache:
// 64 bytes each).  Logits of -inf are left out of all this, or a mask would make
// one long tie of them; where fewer than k others are left the first of them
// follow in order.
constexpr uint32_t kNone = 0x007fffffu;   // order_bits(-inf)
constexpr int kListCap = 2048;            // kMaxTop * max(groups per run, elements per group)
template <int THREADS>
struct TopLds {
  __align__(16) uint64_t list[kListCap];
  uint32_t run[THREADS];      // order bits of the runs' maxima
  uint32_t chosen[kMaxTop];   // the groups
  uint32_t count, bound;
};

typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ int rank_in(uint64_t key, const uint64_t* list, int n) {
  int r = 0, i = 0;
#pragma unroll 4
  for (; i + 2 <= n; i += 2) {
    const u64x2 v = *reinterpret_cast<const u64x2*>(list + i);
    r += (v[0] > key ? 1 : 0) + (v[1] > key ? 1 : 0);
  }
  if (i < n) r += list[i] > key ? 1 : 0;
  return r;
}

// Of a wave's 64 N numbers: an x that at least k of them reach, and that either
// exactly k reach or that is the k-th largest (0 if fewer than k are above 0).
// Bisection over the bits; a step is N ballots.  Stopped at bit LAST, x is
// rounded down: more than k may reach it.
template <int N, int LAST = 0>
__device__ __forceinline__ uint32_t kth_largest(const uint32_t* v, int k) {
  uint32_t x = 0;
  for (int bit = 31; bit >= LAST; --bit) {
    const uint32_t c = x | (1u << bit);
    int n = 0;
#pragma unroll
    for (int q = 0; q < N; ++q) n += __popcll(__ballot(v[q] >= c));
    if (n >= k) x = c;
    if (n == k) break;
  }
  return x;
}

__device__ __forceinline__ uint64_t lanes_below() {
  return (uint64_t(1) << (threadIdx.x & 63)) - 1;
}

// The listed keys by rank, and masked logits to make up the number.
template <bool BF, int THREADS, typename Put>
__device__ __forceinline__ void rank_list(const typename Elem<BF>::T* row, int64_t n, int k,
                                          TopLds<THREADS>& t, Put put) {
  const int tid = threadIdx.x, lane = tid & 63;
  int m = (int)t.count;
  for (int i = tid; i < m; i += THREADS) {
    const uint64_t key = t.list[i];
    const int rank = rank_in(key, t.list, m);
    if (rank < k) put(rank, key);
  }
  if (tid < 64) {
    for (int64_t j0 = 0; m < k && j0 < n; j0 += 64) {
      const bool masked = j0 + lane < n && Elem<BF>::get(row + j0 + lane) == kNegInf;
      const uint64_t mask = __ballot(masked);
      const int rank = m + __popcll(mask & lanes_below());
      if (masked && rank < k) put(rank, order_key(kNegInf, (uint32_t)(j0 + lane)));
      m += __popcll(mask);
    }
  }
}

// Keys of the k first elements of row[0, n), in order, to put(rank, key);
// n >= k.  `group` holds the maxima of groups of G elements.
template <bool BF, int THREADS, typename Put>
__device__ void select_top(const typename Elem<BF>::T* row, int64_t n, const float* group, int k,
                           TopLds<THREADS>& t, Put put) {
  constexpr int G = 4 * Elem<BF>::kN, W = THREADS / 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int ng = (int)((n + G - 1) / G);
  const int run = (ng + THREADS - 1) / THREADS;   // groups per run
  const int g0 = tid * run, g1 = min(ng, g0 + run);
  uint32_t best = 0;
  for (int g = g0; g < g1; ++g) best = max(best, order_bits(group[g]));
  t.run[tid] = best;
  if (tid == 0) t.count = 0;
  __syncthreads();
  // the k best runs, ties by index; every wave finds the same
  uint32_t v[W];
#pragma unroll
  for (int q = 0; q < W; ++q) v[q] = t.run[q * 64 + lane];
  const uint32_t x = max(kth_largest<W>(v, k), kNone + 1);
  int above = 0, before = 0;
#pragma unroll
  for (int q = 0; q < W; ++q) {
    above += __popcll(__ballot(v[q] > x));
    const uint64_t same = __ballot(v[q] == x);
    before += q < wave ? __popcll(same) : q == wave ? __popcll(same & lanes_below()) : 0;
  }
  if (best > x || (best == x && before < k - above)) {
    for (int g = g0; g < g1; ++g) {
      const uint32_t o = order_bits(group[g]);
      if (o >= x) t.list[atomicAdd(&t.count, 1u)] = ((uint64_t)o << 32) | (uint32_t)~(uint32_t)g;
    }
  }
  __syncthreads();
  // the k best groups of those runs
  int m = (int)t.count;
  if (tid == 0) t.bound = x;
  __syncthreads();
  for (int i = tid; i < m; i += THREADS) {
    const uint64_t key = t.list[i];
    const int rank = rank_in(key, t.list, m);
    if (rank < k) t.chosen[rank] = ~(uint32_t)key;
    if (rank == k - 1) t.bound = (uint32_t)(key >> 32);
  }
  const int picked = min(m, k);
  __syncthreads();
  const uint32_t least = t.bound;
  if (tid == 0) t.count = 0;
  __syncthreads();
  // their k best elements
  for (int i = tid; i < picked * G; i += THREADS) {
    const int64_t j = (int64_t)t.chosen[i / G] * G + i % G;
    if (j < n) {
      const uint64_t key = order_key(Elem<BF>::get(row + j), (uint32_t)j);
      if ((uint32_t)(key >> 32) >= least) t.list[atomicAdd(&t.count, 1u)] = key;
    }
  }
  __syncthreads();
  rank_list<BF, THREADS>(row, n, k, t, put);
}

// The same for a chunk that the threads still hold in `raw` (U vectors each, absent
// elements -inf), `most` being the largest of a thread's.  Every wave whose lanes
// all hold elements finds its q-th largest maximum, q = k / (number of such waves)
// rounded up: the least of these is reached by k elements at least, and what
// reaches it is ranked.  Returns false where that is more than kHeldCap (ties, or
// the largest close together), which select_top then settles.
constexpr uint32_t kHeldCap = 512;
template <bool BF, int THREADS, int U, typename Put>
__device__ bool select_held(const typename Elem<BF>::Vec* raw, float most,
                            const typename Elem<BF>::T* row, int64_t n, int k, TopLds<THREADS>& t,
                            Put put) {
  using E = Elem<BF>;
  constexpr int kBits = U * E::kN;
  static_assert(kBits <= 32, "a bit per element");
  const int tid = threadIdx.x, wave = tid >> 6;
  const int full = max(1, min(THREADS / 64, (int)(n / E::kN) / 64));
  if (wave < full) {
    const uint32_t own = order_bits(most);
    // 16 bits are all a bf16 has; 20 of a float32 round down by 2^-11 at most
    const uint32_t x = kth_largest<1, BF ? 16 : 12>(&own, (k + full - 1) / full);
    if ((tid & 63) == 0) t.run[wave] = x;
  }
  if (tid == 0) t.count = 0;
  __syncthreads();
  uint32_t x = t.run[0];
  for (int w = 1; w < full; ++w) x = min(x, t.run[w]);
  const float least = order_value(max(x, kNone + 1));
  uint32_t hits = 0;   // a bit per element; a NaN too
  if (!(most < least)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float z[E::kN];
      E::decode(raw[u], z);
#pragma unroll
      for (int q = 0; q < E::kN; ++q) hits |= (z[q] < least ? 0u : 1u) << (u * E::kN + q);
    }
  }
  // places in the list: the wave's lanes one after the other, one atomic per wave
  const int mine = __popc(hits);
  int before = 0, all = 0;
#pragma unroll
  for (int b = 0; b < 6; ++b) {
    const uint64_t m = __ballot((mine >> b) & 1);
    before += __popcll(m & lanes_below()) << b;
    all += __popcll(m) << b;
  }
  uint32_t slot = 0;
  if ((tid & 63) == 0 && all > 0) slot = atomicAdd(&t.count, (uint32_t)all);
  slot = (uint32_t)__builtin_amdgcn_readfirstlane((int)slot) + before;
  for (; hits; hits &= hits - 1, ++slot) {
    const int bit = __ffs(hits) - 1;
    typename E::Word word = raw[0][0];   // the element's 32 bits, picked in registers
#pragma unroll
    for (int i = 1; i < 4 * U; ++i) word = bit * 4 / E::kN == i ? raw[i / 4][i % 4] : word;
    const uint32_t j = (uint32_t)((bit / E::kN * THREADS + tid) * E::kN + bit % E::kN);
    if (slot < kHeldCap) t.list[slot] = order_key(E::from_word(word, bit), j);
  }
  __syncthreads();
  if (t.count > kHeldCap) return false;
  rank_list<BF, THREADS>(row, n, k, t, put);
  return true;
}

// Chunk blockIdx.x of a row (or, with one chunk, the whole row and its results).
// kU vectors per thread are loaded before the first is used; per element the loop
// costs a subtraction, two products, an exponential, two maxima and two sums.
// bf16 rows that start inside a 32-bit word are loaded from the word's start and
// shifted by an element, the neighbour lane's first word closing the gap (3584 x
// 50257: 69 us against 82 with loads at odd addresses; which thread adds which
// element stays the same, so a row's results do not depend on where it lies).
// TOP: 0 without alternatives; kGroups through the group maxima; kHeld for chunks
// of one batch, which are still in registers when their statistics are known (one
// kernel for both would keep one workgroup less per SIMD: 141 us against 119 at
// 2048 x 131072 bf16, top 20).  PAST: the logits do not fit the last-level cache
// and are loaded past it (3584 x 131072 bf16: 147 us a pass against 172, 6.4 TB/s).
constexpr int kGroups = 1, kHeld = 2;
template <bool BF, int THREADS, int TOP, bool SPLIT, bool PAST>
__global__ __launch_bounds__(THREADS) void dora_logprob_fwd(
    const void* logits, int64_t ld, const int64_t* targets, float* logp, float* entropy, float* lse,
    float* top_logp, int64_t* top_index, Stat* part, uint64_t* part_top, int64_t rows, int64_t V,
    int64_t chunk, int top, float scale) {
  using E = Elem<BF>;
  using T = typename E::T;
  constexpr int kStep = THREADS * E::kN;
  extern __shared__ float group[];
  __shared__ Stat lds[THREADS / 64];
  const float c2 = scale * kLog2e;
  const int64_t lo = (int64_t)blockIdx.x * chunk;
  const int64_t n = min(V - lo, chunk);
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const T* z = reinterpret_cast<const T*>(logits) + row * ld + lo;
    const int64_t own = (int64_t)threadIdx.x * E::kN;
    typename E::Vec raw[kU];
    uint32_t edge[BF ? kU : 1];   // of the last lane: the word after its vector
    // The word before the row's first element is read with it, and the one after a
    // batch's last: never the tensor's ends.
    const bool odd = BF && reinterpret_cast<uintptr_t>(z) % 4 != 0 && (row > 0 || lo > 0);
    auto shifted = [&](int64_t j0) { return odd && n - j0 > kStep * kU; };
    auto load = [&](int64_t j0) {
      if (n - j0 >= kStep * kU) {
        const T* from = z + j0 - (shifted(j0) ? 1 : 0);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const T* at = from + u * kStep + own;
          raw[u] = PAST ? E::raw_past(at) : E::raw(at);
        }
        if constexpr (BF) {
          if (shifted(j0) && (threadIdx.x & 63) == 63) {
#pragma unroll
            for (int u = 0; u < kU; ++u)
              edge[u] = *reinterpret_cast<const uint32_t*>(from + u * kStep + own + E::kN);
          }
        }
      } else {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int64_t j = j0 + u * kStep + own;
          raw[u] = E::masked();
          if (j + E::kN <= n) raw[u] = E::raw(z + j);
        }
      }
    };
    load(0);   // in flight while the target is looked up
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
    const float at = SPLIT ? 0.f : E::get(z + y);
    Stat a = empty_stat();
    auto group_max = [&](const float* v, int64_t j) {
      float m = v[0];
#pragma unroll
      for (int q = 1; q < E::kN; ++q) m = maxnan(m, v[q]);
      m = maxnan(m, dpp_move<0xB1>(m));
      m = maxnan(m, dpp_move<0x4E>(m));
      if ((threadIdx.x & 3) == 0 && j < n) group[j / (4 * E::kN)] = m;
    };
    for (int64_t j0 = 0;;) {
      if (n - j0 >= kStep * kU) {
        if constexpr (BF) {
          if (shifted(j0)) {
#pragma unroll
            for (int u = 0; u < kU; ++u) {
              // wave_shl:1, the last lane keeps its own
              const uint32_t next = (uint32_t)__builtin_amdgcn_update_dpp(
                  (int)edge[u], (int)raw[u][0], 0x130, 0xf, 0xf, false);
#pragma unroll
              for (int d = 0; d < 4; ++d)
                raw[u][d] = __builtin_amdgcn_alignbit(d < 3 ? raw[u][d < 3 ? d + 1 : 3] : next,
                                                      raw[u][d], 16);
            }
          }
        }
        float v[kU][E::kN];
#pragma unroll
        for (int u = 0; u < kU; ++u) E::decode(raw[u], v[u]);
        if (TOP) {
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            if (TOP == kGroups) group_max(v[u], j0 + u * kStep + own);
          }
        }
        add_logits<kU * E::kN>(a, &v[0][0], c2);
      } else {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int64_t j = j0 + u * kStep + own;
          if (j0 + u * kStep >= n) break;
          float v[E::kN];
          E::decode(raw[u], v);
          if (j < n && j + E::kN > n) {
            load_part<BF>(z, j, n, kNegInf, v);
            raw[u] = E::encode(v);
          }
          if (TOP == kGroups) group_max(v, j);
          add_logits<E::kN>(a, v, c2);
        }
      }
      j0 += kStep * kU;
      if (j0 >= n) break;
      load(j0);
    }
    const float most = a.m;
    a = block_stat<THREADS / 64>(a, c2, lds);
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
      __shared__ TopLds<THREADS> lists;
      const int k = (int)min((int64_t)top, n);
      uint64_t* mine = SPLIT ? part_top + (row * gridDim.x + blockIdx.x) * top : nullptr;
      if (SPLIT && k < top && (int)threadIdx.x >= k && (int)threadIdx.x < top)
        mine[threadIdx.x] = 0;   // a chunk shorter than the list
      auto put = [&](int rank, uint64_t key) {
        const uint32_t index = ~(uint32_t)key;
        if (SPLIT) {
          mine[rank] = (key & 0xffffffff00000000ull) | (uint32_t)~(index + (uint32_t)lo);
        } else {
          const float v = order_value((uint32_t)(key >> 32));
          top_index[row * top + rank] = index;
          top_logp[row * top + rank] = out.none ? kNegInf : (v - out.ref) * scale - out.log_s;
        }
      };
      bool done = false;
      if constexpr (TOP == kHeld) {
        done = select_held<BF, THREADS, kU>(raw, most, z, n, k, lists, put);
        if (!done) {
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            float v[E::kN];
            E::decode(raw[u], v);
            group_max(v, u * kStep + own);
          }
        }
      }
      if (!done) {
        __syncthreads();   // the group maxima are complete
        select_top<BF, THREADS>(z, n, group, k, lists, put);
      }
    }
    __syncthreads();   // LDS is written again for the next row
  }
}

// Joins the chunks of a row: their statistics, and the first k of their sorted
// lists.  Every wave takes up to 128 of the lists' foremost keys; what is below
// the k-th of those, or below the last of any one list, is out, and the rest is
// ranked.  The dynamic LDS holds all keys (at most kMaxSplits kMaxTop), which
// many equal logits may leave.
static_assert(kMaxSplits == 64, "a list per lane");
template <bool BF, bool TOP>
__global__ __launch_bounds__(kThreads) void dora_logprob_join(
    const void* logits, int64_t ld, const int64_t* targets, const Stat* part,
    const uint64_t* part_top, int splits, float* logp, float* entropy, float* lse, float* top_logp,
    int64_t* top_index, int64_t rows, int64_t V, int top, float scale) {
  using E = Elem<BF>;
  extern __shared__ __align__(16) uint64_t list[];
  __shared__ uint32_t count;
  const int tid = threadIdx.x, lane = tid & 63;
  const float c2 = scale * kLog2e;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t y = targets[row];
    const Stat* stats = part + row * splits;
    const uint64_t* lists = TOP ? part_top + row * splits * top : nullptr;
    Stat a = empty_stat();
    uint32_t front[2] = {0, 0};
    uint64_t last = 0, early[2] = {0, 0};   // this thread's first keys
    const bool live = y >= 0 && y < V;
    if (live) {
      if (lane < splits) a = stats[lane];
      if (TOP) {
        // the front: the first `deep` keys of every list
        const int deep = min(top, max(1, 128 / splits));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int i = lane + 64 * q;
          if (i < splits * deep)
            front[q] = (uint32_t)(lists[(int64_t)(i / deep) * top + i % deep] >> 32);
        }
        if (lane < splits) last = lists[(int64_t)lane * top + top - 1];
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (tid + q * kThreads < splits * top) early[q] = lists[tid + q * kThreads];
      }
    }
    if (tid == 0) count = 0;
    if (!live) {
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
    const RowOut out = row_out(wave_stat(a, c2), at, scale);
    if (tid == 0) {
      logp[row] = out.logp;
      if (entropy) entropy[row] = out.entropy;
      if (lse) lse[row] = out.lse;
    }
    if (TOP) {
      __syncthreads();   // count is 0
      const uint32_t x = kth_largest<2, 12>(front, top);
      const uint32_t hi = wave_max((uint32_t)(last >> 32));
      const uint32_t low = wave_max((uint32_t)(last >> 32) == hi ? (uint32_t)last : 0u);
      // at least 1: keys of 0 pad short lists
      const uint64_t least = max(max((uint64_t)x << 32, ((uint64_t)hi << 32) | low), (uint64_t)1);
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (early[q] >= least) list[atomicAdd(&count, 1u)] = early[q];
      for (int i = tid + 2 * kThreads; i < splits * top; i += kThreads) {
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
      __syncthreads();
    }
  }
}

// Gradient of a row's chunk blockIdx.x of kBwdU vectors per thread.  The logits are
// loaded before the row's scalars are known; one exponential per element and no
// reduction, so memory bounds it.  THROUGH: the gradient does not fit the
// last-level cache and is stored past it (4096 x 131072 bf16: 319 us a pass against
// 336, 6.3 TB/s; where it fits, its reader finds it there).  A row whose lse is too
// coarse is read again by each of its workgroups (1024 x 131072 bf16, all rows such:
// 1.1 ms against 0.1).
constexpr int kBwdU = 2;
template <bool BF, int THREADS, bool THROUGH>
__global__ __launch_bounds__(THREADS) void dora_logprob_bwd(
    const float* g_logp, const float* g_entropy, const void* logits, int64_t ld,
    const int64_t* targets, const float* lse, const float* entropy, void* grad, int64_t rows,
    int V, float scale) {
  using E = Elem<BF>;
  using T = typename E::T;
  constexpr int kStep = THREADS * E::kN;
  __shared__ Stat lds[THREADS / 64];
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const T* z = reinterpret_cast<const T*>(logits) + row * ld;
    T* gz = reinterpret_cast<T*>(grad) + row * V;
    // the gradient's vectors lie on 16-byte boundaries; the first may start
    // before the row
    const int off = (int)(reinterpret_cast<uintptr_t>(gz) % 16 / sizeof(T));
    const int j0 = (int)(blockIdx.x * kStep * kBwdU + threadIdx.x * E::kN) - off;
    const uint32_t fits = V >= E::kN ? V - E::kN + 1 : 0;
    auto whole = [&](int j) { return (uint32_t)j < fits; };
    auto store = [&](int j, const float* v) {
      if (whole(j)) {
        if (THROUGH)
          E::store_through(gz + j, v);
        else
          E::store(gz + j, v);
      } else {
#pragma unroll
        for (int q = 0; q < E::kN; ++q)
          if (j + q >= 0 && j + q < V) E::put(gz + j + q, v[q]);
      }
    };
    const int64_t y = targets[row];
    if (y < 0 || y >= V) {
      float o[E::kN] = {};
#pragma unroll
      for (int u = 0; u < kBwdU; ++u) store(j0 + u * kStep, o);
      continue;
    }
    typename E::Vec raw[kBwdU];
#pragma unroll
    for (int u = 0; u < kBwdU; ++u)
      if (whole(j0 + u * kStep)) raw[u] = E::raw(z + j0 + u * kStep);
    float ref = 0.f, log_s = lse[row];
    bool zero = false;
    if (!(fabsf(log_s) <= kCoarseLse)) {   // the same for the whole workgroup
      Stat st = empty_stat();
      for (int j = (int)threadIdx.x * E::kN; j < V; j += kStep) {
        float v[E::kN];
        load_part<BF>(z, j, V, kNegInf, v);
        add_logits<E::kN>(st, v, scale * kLog2e);
      }
      const RowOut r = row_out(block_stat<THREADS / 64>(st, scale * kLog2e, lds), 0.f, scale);
      zero = r.none;
      ref = r.ref;
      log_s = r.log_s;
      __syncthreads();   // lds is written again for the next row
    }
    const float a = zero || !g_logp ? 0.f : g_logp[row];
    const float b = zero || !g_entropy ? 0.f : g_entropy[row];
    const float H = g_entropy ? entropy[row] : 0.f;
#pragma unroll
    for (int u = 0; u < kBwdU; ++u) {
      const int j = j0 + u * kStep;
      if (j >= V) break;
      float v[E::kN];
      if (whole(j)) {
        E::decode(raw[u], v);
      } else {
#pragma unroll
        for (int q = 0; q < E::kN; ++q)
          v[q] = j + q >= 0 && j + q < V ? E::get(z + j + q) : kNegInf;
      }
#pragma unroll
      for (int q = 0; q < E::kN; ++q) {
        const float d = fmaf(v[q] - ref, scale, -log_s);
        const float p = __builtin_amdgcn_exp2f(d * kLog2e);
        // p (log p + H) is 0 where p is; d is NaN where a row is lost
        const float inner = p > 0.f ? d + H : 0.f;
        v[q] = -p * fmaf(b, inner, a) * scale;
        if (zero) v[q] = 0.f;
      }
      const int hit = (int)y - j;
      if ((uint32_t)hit < (uint32_t)E::kN) {
#pragma unroll
        for (int q = 0; q < E::kN; ++q)
          if (q == hit) v[q] = fmaf(a, scale, v[q]);
      }
      store(j, v);
    }
  }
}

constexpr int64_t kLimit = int64_t(1) << 31;
constexpr int64_t kMaxVocab = kMaxSplits * kMaxChunk;   // 2^23

bool shape_ok(const dora_logprob_shape& s) {
  return s.rows >= 0 && s.rows < kLimit && s.vocab >= 1 && s.vocab <= kMaxVocab && s.ld >= s.vocab &&
         s.ld < kLimit && s.top >= 0 && s.top <= DORA_LOGPROB_MAX_TOP && s.top <= s.vocab;
}
bool dtype_ok(const dora_logprob_shape& s) { return s.dtype == DORA_F32 || s.dtype == DORA_BF16; }

int check_shape(const dora_logprob_shape* s) {
  if (!s) return DORA_ERR_NULL;
  // (the kernels work with scale log2(e), which passes float32's range from 1.4 2^127 on)
  if (s->reserved != 0 || !(s->scale > 0.f && s->scale < 0x1p127f)) return DORA_ERR_FLAGS;
  if (!dtype_ok(*s)) return DORA_ERR_DTYPE;
  if (!shape_ok(*s)) return DORA_ERR_SHAPE;
  return DORA_OK;
}

// How many workgroups read a row.  With rows enough to give every CU a few
// workgroups each row is one workgroup's; below that rows are cut until about
// kWantBlocks workgroups run, down to chunks of one batch (kU vectors a thread).
constexpr int64_t kWantBlocks = 1024;
struct Plan {
  int64_t chunk, splits;
  size_t stat_bytes, top_bytes;
};
Plan plan(const dora_logprob_shape& s) {
  Plan p;
  const int64_t unit = kThreads * kU * (s.dtype == DORA_BF16 ? 8 : 4);
  // rows of under two batches are not worth the join
  const int64_t batches = s.vocab < 2 * unit ? 1 : (s.vocab + unit - 1) / unit;
  const int64_t most = std::min(kMaxSplits, batches);
  const int64_t want = std::max<int64_t>(1, kWantBlocks / std::max<int64_t>(1, s.rows));
  const int64_t least = (s.vocab + kMaxChunk - 1) / kMaxChunk;
  const int64_t n = std::max(least, std::min(want, most));
  p.chunk = std::min(kMaxChunk, ((s.vocab + n - 1) / n + unit - 1) / unit * unit);
  p.splits = (s.vocab + p.chunk - 1) / p.chunk;
  const int64_t parts = p.splits > 1 ? s.rows * p.splits : 0;
  p.stat_bytes = (size_t)((parts * (int64_t)sizeof(Stat) + 15) / 16 * 16);
  p.top_bytes = (size_t)(parts * s.top * 8);
  return p;
}
// Whether a call's logits pass the last-level cache.
template <bool BF>
bool past_last_level(const dora_logprob_shape& s) {
  constexpr double kLastLevel = 256.0 * (1 << 20);
  return (double)s.rows * (double)s.vocab * sizeof(typename Elem<BF>::T) > kLastLevel;
}

// Short rows are one wave's: no barriers, and four times the rows in flight.
constexpr int64_t kWaveVocab = 4096;

template <bool BF, int THREADS, int TOP, bool SPLIT, bool PAST>
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
    hipLaunchKernelGGL((dora_logprob_fwd<BF, THREADS, TOP, SPLIT, PAST>), dim3((unsigned)p.splits, rows),
                       dim3(THREADS), groups, st, logits, s.ld, targets, logp, entropy, lse,
                       top_logp, top_index, part, part_top, s.rows, s.vocab, p.chunk, (int)s.top,
                       s.scale);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (!SPLIT) return hipSuccess;
  LaunchTimer t("logprob_join", st);
  hipLaunchKernelGGL((dora_logprob_join<BF, (TOP > 0)>), dim3((unsigned)std::min(s.rows, kMaxGrid)),
                     dim3(kThreads), TOP ? (size_t)(p.splits * s.top * 8) : 0, st, logits, s.ld,
                     targets, part, part_top, (int)p.splits, logp, entropy, lse, top_logp,
                     top_index, s.rows, s.vocab, (int)s.top, s.scale);
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
  constexpr int N = kThreads;
  const bool top = s.top > 0, past = past_last_level<BF>(s);
  const int64_t batch = N * kU * Elem<BF>::kN;
  if (p.splits > 1) {
    if (top && p.chunk <= batch) return go(launch_fwd<BF, N, kHeld, true, false>);
    if (top)
      return past ? go(launch_fwd<BF, N, kGroups, true, true>)
                  : go(launch_fwd<BF, N, kGroups, true, false>);
    return past ? go(launch_fwd<BF, N, 0, true, true>) : go(launch_fwd<BF, N, 0, true, false>);
  }
  if (s.vocab <= kWaveVocab) {
    if (!top) return go(launch_fwd<BF, 64, 0, false, false>);
    return s.vocab <= batch / 4 ? go(launch_fwd<BF, 64, kHeld, false, false>)
                                : go(launch_fwd<BF, 64, kGroups, false, false>);
  }
  if (top && s.vocab <= batch) return go(launch_fwd<BF, N, kHeld, false, false>);
  if (top)
    return past ? go(launch_fwd<BF, N, kGroups, false, true>)
                : go(launch_fwd<BF, N, kGroups, false, false>);
  return past ? go(launch_fwd<BF, N, 0, false, true>) : go(launch_fwd<BF, N, 0, false, false>);
}

template <bool BF>
hipError_t backward(const dora_logprob_shape& s, const float* g_logp, const float* g_entropy,
                    const void* logits, const int64_t* targets, const float* lse,
                    const float* entropy, void* grad, hipStream_t st) {
  LaunchTimer t("logprob_bwd", st);
  auto launch = [&](auto kernel, int threads) {
    const int64_t per = (int64_t)threads * Elem<BF>::kN * kBwdU;
    hipLaunchKernelGGL(kernel,   // a row may take one vector more than its elements fill
                       dim3((unsigned)((s.vocab + Elem<BF>::kN - 1 + per - 1) / per),
                            (unsigned)std::min<int64_t>(s.rows, 65535)),
                       dim3(threads), 0, st, g_logp, g_entropy, logits, s.ld, targets, lse, entropy,
                       grad, s.rows, (int)s.vocab, s.scale);
    return hipGetLastError();
  };
  if (past_last_level<BF>(s)) return launch(dora_logprob_bwd<BF, kThreads, true>, kThreads);
  if (s.vocab <= kWaveVocab) return launch(dora_logprob_bwd<BF, 64, false>, 64);
  return launch(dora_logprob_bwd<BF, kThreads, false>, kThreads);
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
