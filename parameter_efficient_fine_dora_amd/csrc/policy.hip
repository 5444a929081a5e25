// Clipped policy loss with a divergence from a reference, and its gradient.
//
//   rho = exp(logp - old), gain = A min(rho, 1 + hi) or A min(max(rho, 1 - lo), dual) by A's sign,
//   kl = exp(d) - 1 - d with d = ref - logp, l = -gain + kl_coef kl
//
// Both directions read 13 to 17 bytes a token and do two exponentials; the gradient
// writes four.  Memory bounds large batches, launches small ones.  The terms are
// float64: whether a bound holds a ratio must not depend on a float32 rounding beside
// the bound (the slope jumps there), the loss is a small difference of large sums, and
// exp(d) - 1 - d cancels.  The exponentials are the library's: a Taylor sum of the same precision, to
// r^13 with log 2 in two parts, takes as long, one to r^10 1.5 us less of 4.2M tokens' gradient but is 2.4e-13
// off.  That gradient takes 18.6 us (4.7 TB/s); 1M packed tokens' loss is 13 us of sums and 8 of joining and
// finishing.
#include <algorithm>
#include <cmath>

#include "checks.h"
#include "kernels.h"
#include "sequences.h"

namespace dora {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kFinish = 1024;
constexpr int64_t kSmallTokens = 4096, kSmallSequences = 32;   // what one workgroup does alone

struct Tokens {
  const float *logp, *old, *ref, *adv;
  double low, high, dual, kl_coef;   // bounds of the ratio: 1 - clip_low, 1 + clip_high
};

struct Term {
  double loss, slope, kl, held, ratio;
};

__device__ __forceinline__ Term term(const Tokens& k, float logp, float old, float ref, float adv) {
  Term x;
  const double a = adv;
  x.ratio = exp((double)logp - (double)old);
  const bool over = a > 0.0 ? x.ratio > k.high : a < 0.0 && x.ratio > k.dual;
  const bool under = a < 0.0 && x.ratio < k.low;
  const double bounded = over ? (a > 0.0 ? k.high : k.dual) : under ? k.low : x.ratio;
  x.held = over || under ? 1.0 : 0.0;
  // an advantage of 0 gives 0 whatever the ratio (an infinite one too, where it has an upper bound)
  x.loss = a == 0.0 && x.ratio > k.high ? 0.0 : -a * bounded;
  x.slope = over || under || (a == 0.0 && x.ratio > k.high) ? 0.0 : -a * x.ratio;
  x.kl = 0.0;
  if (k.ref) {
    const double d = (double)ref - (double)logp, e = expm1(d);
    x.kl = e < INFINITY ? e - d : e;   // an infinite d is nothing beside its exponential; NaN stays
    if (k.kl_coef > 0.0) {
      x.loss += k.kl_coef * x.kl;
      x.slope -= k.kl_coef * e;
    }
  }
  return x;
}

__device__ __forceinline__ int64_t wave_id() {
  return (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// A round's four tokens of a lane: their values, which of them count, and the factor
// or advantage of their sequences.
struct Four {
  bool live[4];
  float logp[4], old[4], ref[4], adv[4];
  __device__ __forceinline__ void load(const Batch& b, const Tokens& k, int64_t t, bool each) {
    counted(b, t, live);
    load4(k.logp, t, b.tokens, logp);
    load4(k.old, t, b.tokens, old);
    if (k.ref) load4(k.ref, t, b.tokens, ref);
    if (each) load4(k.adv, t, b.tokens, adv);
  }
};

constexpr int kTotals = 5;   // loss, counted, kl, held, ratio

// Sums over chunk w, by a wave: its totals in `totals` (LDS); SEQ: also the loss and count of each
// sequence.
template <bool SEQ, bool PER>
__device__ __forceinline__ void chunk_sums(const Batch& b, const Parts& parts, int64_t chunk, int64_t w,
                                           const Tokens& k, double* totals) {
  const int64_t c0 = min(w * chunk, b.tokens);
  const int64_t c1 = min(c0 + chunk, b.tokens);
  const int lane = threadIdx.x & 63;
  Four x;   // loads are under way while the sequence is looked for, and a round ahead
  x.load(b, k, c0 + lane * 4, !PER);
  Cursor at = cursor_at(b, c0);
  Pair64 sum = {0.0, 0.0};
  double all[kTotals] = {};
  auto give = [&](Pair64* to) {
    const Pair64 x = {wave_sum64(sum.v), wave_sum64(sum.n)};
    if (lane == 0) *to = x;
    sum = {0.0, 0.0};
  };
  for (int64_t r0 = c0; r0 < c1; r0 += kRound) {
    const int64_t t = r0 + lane * 4, r1 = min(r0 + kRound, c1);
    Four ahead;
    if (r1 < c1) ahead.load(b, k, t + kRound, !PER);
    // tokens of no sequence do not count; the others get their sequence's advantage
    bool real[4] = {};
    Cursor look = at;
    through_round(
        b, look, r0, r1, c1,
        [&](int64_t s, int64_t from, int64_t to) {
          const float a = PER ? k.adv[s] : 0.f;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (t + q >= from && t + q < to) {
              real[q] = x.live[q];
              if (PER) x.adv[q] = a;
            }
          }
        },
        [](int64_t, bool) {});
    double loss[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      loss[q] = 0.0;
      if (real[q]) {
        const Term v = term(k, x.logp[q], x.old[q], x.ref[q], x.adv[q]);
        loss[q] = v.loss;
        all[0] += v.loss;
        all[1] += 1.0;
        all[2] += v.kl;
        all[3] += v.held;
        all[4] += v.ratio;
      }
    }
    if (SEQ)
      through_round(
          b, at, r0, r1, c1,
          [&](int64_t, int64_t from, int64_t to) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (real[q] && t + q >= from && t + q < to) {
                sum.v += loss[q];
                sum.n += 1.0;
              }
            }
          },
          [&](int64_t s, bool began) { give(began ? parts.own + s : parts.head + w); });
    at = look;
    x = ahead;
  }
  if (SEQ && c0 < c1 && b.inside(at.s)) give(at.began ? parts.tail + w : parts.head + w);
#pragma unroll
  for (int i = 0; i < kTotals; ++i) {
    const double v = wave_sum64(all[i]);
    if (lane == 0) totals[i] = v;
  }
}

template <bool SEQ, bool PER>
__global__ __launch_bounds__(kThreads) void dora_policy_sums(const Batch b, const Parts parts,
                                                             int64_t chunk, const Tokens k,
                                                             double* totals) {
  __shared__ double lds[kWaves][kTotals];
  chunk_sums<SEQ, PER>(b, parts, chunk, wave_id(), k, lds[threadIdx.x >> 6]);
  __syncthreads();
  if (threadIdx.x < kTotals) {
    const int i = threadIdx.x;
    totals[(int64_t)blockIdx.x * kTotals + i] = (lds[0][i] + lds[1][i]) + (lds[2][i] + lds[3][i]);
  }
}
static_assert(kWaves == 4, "four waves' totals are added");

// Each sequence's mean and count, in place of its sums, a wave per sequence.
__device__ __forceinline__ void join_means(const Batch& b, const Parts& parts, int64_t chunk, int64_t first,
                                           int64_t waves) {
  for (int64_t s = first; s < b.sequences; s += waves) {
    const Pair64 x = join(b, parts, s, chunk);
    if ((threadIdx.x & 63) == 0) parts.own[s] = {x.n > 0.0 ? x.v / x.n : 0.0, x.n};
  }
}

__global__ __launch_bounds__(kThreads) void dora_policy_join(const Batch b, const Parts parts,
                                                             int64_t chunk) {
  join_means(b, parts, chunk, wave_id(), (int64_t)gridDim.x * kWaves);
}

// Sums of N values over the workgroup's 16 waves, to every thread.
template <int N>
__device__ __forceinline__ void finish_sum(double* v, double* lds) {
  static_assert(kFinish == 16 * 64, "a row of 16 lanes has a wave's sum each");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = wave_sum64(v[i]);
    if ((threadIdx.x & 63) == 0) lds[i * 16 + (threadIdx.x >> 6)] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane_value64(row_sum64(lds[i * 16 + (threadIdx.x & 15)]), 0);
  __syncthreads();
}

// The loss, the statistics and the factors, by one workgroup, from `groups` totals.
struct Results {
  double denominator;
  float *loss, *stats, *weight;
};
template <bool SEQ>
__device__ __forceinline__ void finish(int64_t sequences, const Pair64* means, const double* totals,
                                       int64_t groups, const Results& to, double* lds) {
  double all[kTotals] = {};
  for (int64_t c = threadIdx.x; c < groups; c += kFinish) {
#pragma unroll
    for (int i = 0; i < kTotals; ++i) all[i] += totals[c * kTotals + i];
  }
  finish_sum<kTotals>(all, lds);
  double sum[2] = {all[0], all[1]};   // of the losses, and how many of them
  if (SEQ) {
    sum[0] = sum[1] = 0.0;
    for (int64_t s = threadIdx.x; s < sequences; s += kFinish) {
      sum[0] += means[s].v;
      sum[1] += means[s].n > 0.0 ? 1.0 : 0.0;
    }
    finish_sum<2>(sum, lds);
  }
  const double by = to.denominator > 0.0 ? to.denominator : fmax(sum[1], 1.0);
  if (SEQ) {
    for (int64_t s = threadIdx.x; s < sequences; s += kFinish)
      to.weight[s] = means[s].n > 0.0 ? (float)(1.0 / (means[s].n * by)) : 0.f;
  }
  if (threadIdx.x == 0) {
    const double n = fmax(all[1], 1.0);
    *to.loss = (float)(sum[0] / by);
    if (!SEQ) *to.weight = (float)(1.0 / by);
    to.stats[0] = (float)(all[2] / n);
    to.stats[1] = (float)(all[3] / n);
    to.stats[2] = (float)(all[4] / n);
    to.stats[3] = (float)all[1];
  }
}
template <bool SEQ>
__global__ __launch_bounds__(kFinish) void dora_policy_finish(int64_t sequences, const Pair64* means,
                                                              const double* totals, int64_t groups,
                                                              const Results to) {
  __shared__ double lds[kFinish / 64 * kTotals];
  finish<SEQ>(sequences, means, totals, groups, to, lds);
}
// All of a small batch's loss by one workgroup, a round a wave: one launch (from Python eight answers of
// 256 tokens 7.4 us, in two launches 9.2; of 512 9.3 and 9.2; of 1024, two rounds a wave, 13.7 and
// 9.2; means of 64 sequences of 32 20.3 and 19.2).
template <bool SEQ, bool PER>
__global__ __launch_bounds__(kFinish) void dora_policy_small(const Batch b, const Parts parts, int64_t chunk,
                                                             const Tokens k, const Results to) {
  __shared__ double totals[kFinish / 64 * kTotals], lds[kFinish / 64 * kTotals];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  chunk_sums<SEQ, PER>(b, parts, chunk, wave, k, totals + wave * kTotals);
  __syncthreads();   // the workgroup's own writes are there
  if (SEQ) {
    join_means(b, parts, chunk, wave, kFinish / 64);
    __syncthreads();
  }
  finish<SEQ>(b.sequences, parts.own, totals, kFinish / 64, to, lds);
}

template <bool SEQ, bool PER>
__global__ __launch_bounds__(kThreads) void dora_policy_grad(const Batch b, int64_t chunk,
                                                             const Tokens k, const float* grad_loss,
                                                             const float* weight, float* grad) {
  const int64_t c0 = wave_id() * chunk;
  if (c0 >= b.tokens) return;
  const int64_t c1 = min(c0 + chunk, b.tokens);
  const double g = *grad_loss, flat = SEQ ? 0.0 : g * (double)*weight;
  Four x;   // under way while the sequence is looked for
  x.load(b, k, c0 + (threadIdx.x & 63) * 4, !PER);
  Cursor at = cursor_at(b, c0);
  for (int64_t r0 = c0; r0 < c1; r0 += kRound) {
    const int64_t t = r0 + (threadIdx.x & 63) * 4;
    if (r0 > c0) x.load(b, k, t, !PER);
    bool real[4] = {};
    double factor[4] = {};
    through_round(
        b, at, r0, min(r0 + kRound, c1), c1,
        [&](int64_t s, int64_t from, int64_t to) {
          const float a = PER ? k.adv[s] : 0.f;
          const double f = SEQ ? g * (double)weight[s] : flat;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (t + q >= from && t + q < to) {
              real[q] = x.live[q];
              factor[q] = f;
              if (PER) x.adv[q] = a;
            }
          }
        },
        [](int64_t, bool) {});
    float out[4] = {};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (real[q])
        out[q] = (float)(factor[q] * term(k, x.logp[q], x.old[q], x.ref[q], x.adv[q]).slope);
    store_part<false>(grad, t, b.tokens, out);
  }
}

// ---- host ---------------------------------------------------------------------------
unsigned wave_grid(int64_t waves) {
  return (unsigned)std::min<int64_t>((waves + kWaves - 1) / kWaves, int64_t(1) << 20);
}

struct Layout {
  int64_t chunk, chunks;
  size_t tail, own, totals, bytes;
};
Layout layout(const dora_token_batch& b, const dora_policy_options& o) {
  Layout l;
  const bool seq = o.reduce == DORA_REDUCE_SEQUENCE;
  const size_t part = seq ? sizeof(Pair64) : 0;
  l.chunk = chunk_of(b.tokens, kMostSums);
  l.chunks = chunks_of(b.tokens, kMostSums);
  l.tail = (size_t)l.chunks * part;
  l.own = l.tail + (size_t)l.chunks * part;
  l.totals = l.own + (size_t)b.sequences * part;
  l.bytes = l.totals + (size_t)wave_grid(l.chunks) * kTotals * sizeof(double);
  return l;
}

int check_options(const dora_policy_options* o) {
  if (!o) return DORA_ERR_NULL;
  if (!(o->clip_low >= 0 && o->clip_low <= 1) || !(o->clip_high >= 0) || !(o->dual_clip >= 1) ||
      !std::isfinite(o->kl_coef) || o->kl_coef < 0 || !std::isfinite(o->denominator) ||
      o->denominator < 0 || (o->reduce != DORA_REDUCE_TOKEN && o->reduce != DORA_REDUCE_SEQUENCE) ||
      (o->per_sequence != 0 && o->per_sequence != 1))
    return DORA_ERR_FLAGS;
  return DORA_OK;
}

Tokens tokens_of(const dora_policy_options& o, const float* logp, const float* old, const float* ref,
                 const float* adv) {
  return {logp, old, ref, adv, 1.0 - o.clip_low, 1.0 + o.clip_high, o.dual_clip, o.kl_coef};
}

// fn(sequence?, per-sequence advantages?) with both as constants.
template <typename Fn>
void by_options(const dora_policy_options& o, Fn fn) {
  const bool seq = o.reduce == DORA_REDUCE_SEQUENCE, per = o.per_sequence == 1;
  if (seq && per) return fn(std::true_type(), std::true_type());
  if (seq) return fn(std::true_type(), std::false_type());
  if (per) return fn(std::false_type(), std::true_type());
  fn(std::false_type(), std::false_type());
}

}  // namespace
}  // namespace dora

using namespace dora;

extern "C" {

DORA_API size_t dora_policy_workspace_bytes(const dora_token_batch* batch,
                                            const dora_policy_options* options) {
  if (check_batch(batch) != DORA_OK || check_options(options) != DORA_OK) return 0;
  return layout(*batch, *options).bytes;
}

DORA_API int dora_policy_forward(const dora_token_batch* batch, const dora_policy_options* options,
                                 const float* logp, const float* old_logp, const float* ref_logp,
                                 const float* advantages, float* loss, float* stats, float* weight,
                                 void* ws, size_t ws_bytes, void* hip_stream) {
  DORA_CHECK(check_batch(batch));
  DORA_CHECK(check_options(options));
  const bool none = batch->tokens == 0, seq = options->reduce == DORA_REDUCE_SEQUENCE;
  const bool no_seq = batch->sequences == 0;
  DORA_CHECK(check_elem(logp, 4, none));
  DORA_CHECK(check_elem(old_logp, 4, none));
  DORA_CHECK(check_elem(ref_logp, 4, true));
  DORA_CHECK(check_elem(advantages, 4, none || (options->per_sequence && no_seq)));
  DORA_CHECK(check_elem(loss, 4, false));
  DORA_CHECK(check_elem(stats, 4, false));
  DORA_CHECK(check_elem(weight, 4, seq && no_seq));
  const Layout l = layout(*batch, *options);
  DORA_CHECK(check_ws(ws, ws_bytes, l.bytes));
  const Batch b = device_batch(*batch);
  uint8_t* p = reinterpret_cast<uint8_t*>(ws);
  const Parts parts = {reinterpret_cast<Pair64*>(p), reinterpret_cast<Pair64*>(p + l.tail),
                       reinterpret_cast<Pair64*>(p + l.own)};
  double* totals = reinterpret_cast<double*>(p + l.totals);
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  const Tokens k = tokens_of(*options, logp, old_logp, ref_logp, advantages);
  const Results to = {options->denominator, loss, stats, weight};
  if (b.tokens <= kSmallTokens && (!seq || b.sequences <= kSmallSequences)) {
    LaunchTimer timer("policy_small", st);
    by_options(*options, [&](auto seq_, auto per_) {
      hipLaunchKernelGGL((dora_policy_small<decltype(seq_)::value, decltype(per_)::value>), dim3(1),
                         dim3(kFinish), 0, st, b, parts, chunk_of(b.tokens, kFinish / 64), k, to);
    });
    HIP_TRY(hipGetLastError());
    return DORA_OK;
  }
  if (!none) {
    LaunchTimer timer("policy_sums", st);
    by_options(*options, [&](auto seq_, auto per_) {
      hipLaunchKernelGGL((dora_policy_sums<decltype(seq_)::value, decltype(per_)::value>),
                         dim3(wave_grid(l.chunks)), dim3(kThreads), 0, st, b, parts, l.chunk, k,
                         totals);
    });
    HIP_TRY(hipGetLastError());
  }
  if (seq && !no_seq) {
    LaunchTimer timer("policy_join", st);
    hipLaunchKernelGGL(dora_policy_join, dim3(wave_grid(b.sequences)), dim3(kThreads), 0, st, b,
                       parts, l.chunk);
    HIP_TRY(hipGetLastError());
  }
  LaunchTimer timer("policy_finish", st);
  auto kernel = seq ? dora_policy_finish<true> : dora_policy_finish<false>;
  hipLaunchKernelGGL(kernel, dim3(1), dim3(kFinish), 0, st, b.sequences, parts.own, totals,
                     (int64_t)(none ? 0 : wave_grid(l.chunks)), to);
  HIP_TRY(hipGetLastError());
  return DORA_OK;
}

DORA_API int dora_policy_backward(const dora_token_batch* batch, const dora_policy_options* options,
                                  const float* grad_loss, const float* weight, const float* logp,
                                  const float* old_logp, const float* ref_logp,
                                  const float* advantages, float* grad_logp, void* hip_stream) {
  DORA_CHECK(check_batch(batch));
  DORA_CHECK(check_options(options));
  const bool none = batch->tokens == 0, seq = options->reduce == DORA_REDUCE_SEQUENCE;
  const bool no_seq = batch->sequences == 0;
  DORA_CHECK(check_elem(grad_loss, 4, none));
  DORA_CHECK(check_elem(weight, 4, none || (seq && no_seq)));
  DORA_CHECK(check_elem(logp, 4, none));
  DORA_CHECK(check_elem(old_logp, 4, none));
  DORA_CHECK(check_elem(ref_logp, 4, true));
  DORA_CHECK(check_elem(advantages, 4, none || (options->per_sequence && no_seq)));
  DORA_CHECK(check_elem(grad_logp, 4, none));
  if (none) return DORA_OK;
  const Batch b = device_batch(*batch);
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  LaunchTimer timer("policy_grad", st);
  const Tokens k = tokens_of(*options, logp, old_logp, ref_logp, advantages);
  const int64_t chunk = chunk_of(b.tokens, kMostGrads);
  by_options(*options, [&](auto seq_, auto per_) {
    hipLaunchKernelGGL((dora_policy_grad<decltype(seq_)::value, decltype(per_)::value>),
                       dim3(wave_grid(chunks_of(b.tokens, kMostGrads))), dim3(kThreads), 0, st, b, chunk, k,
                       grad_loss, weight, grad_logp);
  });
  HIP_TRY(hipGetLastError());
  return DORA_OK;
}

}  // extern "C"
