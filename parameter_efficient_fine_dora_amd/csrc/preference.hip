// Preference loss over pairs of sequences and its gradient.
//
//   score_s = beta sum_t m_t (logp_t - ref_t) [/ count_s],  h = score_c - score_w - margin
//   dL/dlogp_t = m_t beta [/ count_s] sum_p +- grad_loss_p dL/dh_p   over the pairs of its sequence
//
// Nine bytes a token are read forward (two log probabilities and the mask), one is
// read and four are written backward, so a large batch is bound by memory and a
// small one by its launches: two forward (sums of chunks; sequences joined and pairs
// finished), or one where a workgroup does both, and one backward, or two (a
// coefficient per sequence; the tokens).  Scores are differences of sums over
// thousands of tokens, so sums are float64.
#include <algorithm>
#include <cmath>

#include "checks.h"
#include "kernels.h"
#include "sequences.h"

namespace dora {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kSmall = 1024;   // threads of a small batch's workgroup, and what it takes: tokens, and
constexpr int64_t kSmallTokens = 16384, kSmallRows = 32;   // sequences and pairs together

__device__ __forceinline__ int64_t wave_id() {
  return (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// Sums of logp - ref and the counted tokens of chunk w, by a wave.
template <bool REF>
__device__ __forceinline__ void chunk_sums(const Batch& b, const Parts& parts, int64_t chunk, int64_t w,
                                           const float* logp, const float* ref) {
  const int64_t c0 = w * chunk;
  if (c0 >= b.tokens) return;
  const int64_t c1 = min(c0 + chunk, b.tokens);
  const int lane = threadIdx.x & 63;
  bool live[4];
  float l[4], r[4] = {};
  auto load = [&](int64_t t) {
    counted(b, t, live);
    load4(logp, t, b.tokens, l);
    if (REF) load4(ref, t, b.tokens, r);
  };
  load(c0 + lane * 4);   // under way while the sequence is looked for
  Cursor at = cursor_at(b, c0);
  Pair64 sum = {0.0, 0.0};
  auto give = [&](Pair64* to) {
    const Pair64 x = {wave_sum64(sum.v), wave_sum64(sum.n)};
    if (lane == 0) *to = x;
    sum = {0.0, 0.0};
  };
  for (int64_t r0 = c0; r0 < c1; r0 += kRound) {
    const int64_t t = r0 + lane * 4;
    if (r0 > c0) load(t);
    through_round(
        b, at, r0, min(r0 + kRound, c1), c1,
        [&](int64_t, int64_t from, int64_t to) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (live[q] && t + q >= from && t + q < to) {
              sum.v += (double)l[q] - (double)r[q];
              sum.n += 1.0;
            }
          }
        },
        [&](int64_t s, bool began) { give(began ? parts.own + s : parts.head + w); });
  }
  if (b.inside(at.s)) give(at.began ? parts.tail + w : parts.head + w);
}

struct Numbers {
  double beta, margin, smoothing;
  int kind;
  bool normalize;
};

__device__ __forceinline__ double softplus(double v) { return fmax(v, 0.0) + log1p(exp(-fabs(v))); }

__device__ __forceinline__ double score_of(const Numbers& o, const Pair64& x) {
  return o.beta * (o.normalize ? x.v / fmax(x.n, 1.0) : x.v);
}

struct Results {
  int64_t pairs;
  const int64_t *chosen, *rejected;
  float *loss, *score, *logit, *count;
};
// A wave per sequence writes its score and count, and one per pair the loss: those from `first` on, each
// `waves`th.
__device__ __forceinline__ void finish(const Batch& b, const Parts& parts, int64_t chunk, const Numbers& o,
                                       const Results& to, int64_t first, int64_t waves) {
  const int lane = threadIdx.x & 63;
  for (int64_t w = first; w < b.sequences + to.pairs; w += waves) {
    if (w < b.sequences) {
      const Pair64 x = join(b, parts, w, chunk);
      if (lane == 0) {
        to.score[w] = (float)score_of(o, x);
        to.count[w] = (float)x.n;
      }
      continue;
    }
    const int64_t p = w - b.sequences, c = to.chosen[p], r = to.rejected[p];
    float out = 0.f, at = 0.f;
    if (b.inside(c) && b.inside(r)) {
      const double h = score_of(o, join(b, parts, c, chunk)) -
                       score_of(o, join(b, parts, r, chunk)) - o.margin;
      double v;
      if (o.kind == DORA_PREFERENCE_SIGMOID) {
        // a term without weight is left out: at an infinite h it would be 0 inf
        v = o.smoothing < 1.0 ? (1.0 - o.smoothing) * softplus(-h) : 0.0;
        if (o.smoothing > 0.0) v += o.smoothing * softplus(h);
      } else if (o.kind == DORA_PREFERENCE_HINGE) {
        v = h >= 1.0 ? 0.0 : 1.0 - h;
      } else {
        v = (h - 0.5) / o.beta;
        v *= v;
      }
      out = (float)v;
      at = (float)h;
    }
    if (lane == 0) {
      to.loss[p] = out;
      to.logit[p] = at;
    }
  }
}

template <bool REF>
__global__ __launch_bounds__(kThreads) void dora_preference_sums(const Batch b, const Parts parts,
                                                                 int64_t chunk, const float* logp,
                                                                 const float* ref) {
  chunk_sums<REF>(b, parts, chunk, wave_id(), logp, ref);
}
__global__ __launch_bounds__(kThreads) void dora_preference_pairs(const Batch b, const Parts parts,
                                                                  int64_t chunk, const Numbers o,
                                                                  const Results to) {
  finish(b, parts, chunk, o, to, wave_id(), (int64_t)gridDim.x * kWaves);
}
// Both for a small batch by one workgroup, a chunk a wave: one launch (from Python a pair of 512 tokens
// each 6.3 us, in two launches 10.0; 8 pairs of 1024 7.7 and 10.1; but 4 pairs of 4096 10.4 and 10.3,
// 32 pairs of 256 15.4 and 10.3).
template <bool REF>
__global__ __launch_bounds__(kSmall) void dora_preference_small(const Batch b, const Parts parts,
                                                                int64_t chunk, const float* logp,
                                                                const float* ref, const Numbers o,
                                                                const Results to) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  chunk_sums<REF>(b, parts, chunk, wave, logp, ref);
  __syncthreads();   // the workgroup's own writes are there
  finish(b, parts, chunk, o, to, wave, kSmall / 64);
}

__device__ __forceinline__ double slope_of(const Numbers& o, double h) {
  if (o.kind == DORA_PREFERENCE_SIGMOID) return o.smoothing - 1.0 / (1.0 + exp(h));
  if (o.kind == DORA_PREFERENCE_HINGE) return h >= 1.0 ? 0.0 : h < 1.0 ? -1.0 : h;
  return 2.0 * (h - 0.5) / (o.beta * o.beta);
}

// What the tokens of sequence s get: its pairs' slopes, looked for in all of them by a whole wave,
// and summed in a fixed order.
struct Pairs {
  Numbers o;
  int64_t count;
  const float *grad_loss, *logit, *counted;
  const int64_t *chosen, *rejected;
};
__device__ __forceinline__ double coefficient(const Batch& b, const Pairs& p, int64_t s) {
  double sum = 0.0;
  for (int64_t i = threadIdx.x & 63; i < p.count; i += 64) {
    const int64_t c = p.chosen[i], r = p.rejected[i];
    const double sign = (c == s ? 1.0 : 0.0) - (r == s ? 1.0 : 0.0);
    if (sign != 0.0 && b.inside(c) && b.inside(r))
      sum += sign * (double)p.grad_loss[i] * slope_of(p.o, p.logit[i]);
  }
  return p.o.beta * wave_sum64(sum) / (p.o.normalize ? fmax((double)p.counted[s], 1.0) : 1.0);
}

// A wave per sequence: many pairs are looked through once for each, and not by each of its waves.
__global__ __launch_bounds__(kThreads) void dora_preference_coef(const Batch b, const Pairs p,
                                                                 double* coef) {
  const int64_t waves = (int64_t)gridDim.x * kWaves;
  for (int64_t s = wave_id(); s < b.sequences; s += waves) {
    const double v = coefficient(b, p, s);
    if ((threadIdx.x & 63) == 0) coef[s] = v;
  }
}

// KNOWN: the coefficients are in coef; else the wave looks for each that it needs.
template <bool KNOWN>
__global__ __launch_bounds__(kThreads) void dora_preference_grad(const Batch b, int64_t chunk,
                                                                 const Pairs p, const double* coef,
                                                                 float* grad) {
  const int64_t c0 = wave_id() * chunk;
  if (c0 >= b.tokens) return;
  const int64_t c1 = min(c0 + chunk, b.tokens);
  Cursor at = cursor_at(b, c0);
  int64_t of = -1;
  float v = 0.f;
  for (int64_t r0 = c0; r0 < c1; r0 += kRound) {
    const int64_t t = r0 + (threadIdx.x & 63) * 4;
    bool live[4];
    float g[4] = {};
    counted(b, t, live);
    through_round(
        b, at, r0, min(r0 + kRound, c1), c1,
        [&](int64_t s, int64_t from, int64_t to) {
          if (s != of) v = (float)(KNOWN ? coef[s] : coefficient(b, p, s));
          of = s;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (live[q] && t + q >= from && t + q < to) g[q] = v;
        },
        [](int64_t, bool) {});
    store_part<false>(grad, t, b.tokens, g);
  }
}

// ---- host ---------------------------------------------------------------------------
struct Layout {
  int64_t chunk, chunks;
  size_t head, tail, own, bytes;
};
Layout layout(const dora_token_batch& b) {
  Layout l;
  l.chunk = chunk_of(b.tokens, kMostSums);
  l.chunks = chunks_of(b.tokens, kMostSums);
  l.head = 0;
  l.tail = l.head + (size_t)l.chunks * sizeof(Pair64);
  l.own = l.tail + (size_t)l.chunks * sizeof(Pair64);
  l.bytes = l.own + (size_t)b.sequences * sizeof(Pair64);   // the coefficients fit there too
  return l;
}
Parts parts_at(const Layout& l, void* ws) {
  uint8_t* p = reinterpret_cast<uint8_t*>(ws);
  return {reinterpret_cast<Pair64*>(p + l.head), reinterpret_cast<Pair64*>(p + l.tail),
          reinterpret_cast<Pair64*>(p + l.own)};
}
unsigned wave_grid(int64_t waves) {
  return (unsigned)std::min<int64_t>((waves + kWaves - 1) / kWaves, int64_t(1) << 20);
}

int check_options(const dora_preference_options* o) {
  if (!o) return DORA_ERR_NULL;
  if (o->kind < DORA_PREFERENCE_SIGMOID || o->kind > DORA_PREFERENCE_SQUARE ||
      (o->normalize != 0 && o->normalize != 1) || !std::isfinite(o->beta) || o->beta <= 0 ||
      !std::isfinite(o->margin) || !(o->smoothing >= 0 && o->smoothing <= 1))
    return DORA_ERR_FLAGS;
  return DORA_OK;
}
int check_pairs(int64_t pairs) {
  return pairs < 0 || pairs >= kMaxSequences ? DORA_ERR_SHAPE : DORA_OK;
}
// Whether a launch of its own looks for every sequence's coefficient.  Otherwise each wave looks through all
// pairs, 64 at a time, for each sequence that its round of tokens meets, which is less than another launch
// for up to eight such looks: of 256 pairs and 512 sequences of 8, 32, 64 and 128 tokens, 128, 32, 16
// and 8 looks, the waves' own take 44, 13.3, 8.1 and 5.7 us, the launch 21.3, 9.4, 8.5 and 8.5; of 64 sequences
// of 64 and 128 tokens 13.9 and 8.8, the launch 9.1 and 8.5; of 4 pairs of 8 sequences of 16 and 64 tokens, 16
// and 4 looks, 9.5 and 6.0, the launch 7.9 and 7.6.  Many pairs are looked through once for a sequence, however
// many waves it has (127 pairs of 2 x 1031 tokens: loss and gradient 19.5 us in all, with the launch 22.8).
constexpr int64_t kMostLooks = 8, kMostPairs = 256;
bool looks_first(const Batch& b, int64_t pairs) {
  const int64_t each = (pairs + 63) / 64;
  return pairs > kMostPairs || (double)b.sequences * kRound * each > (double)kMostLooks * b.tokens;
}
Numbers numbers(const dora_preference_options& o) {
  return {o.beta, o.margin, o.smoothing, o.kind, o.normalize == 1};
}

}  // namespace
}  // namespace dora

using namespace dora;

extern "C" {

DORA_API size_t dora_preference_workspace_bytes(const dora_token_batch* batch) {
  return check_batch(batch) == DORA_OK ? layout(*batch).bytes : 0;
}

DORA_API int dora_preference_forward(const dora_token_batch* batch,
                                     const dora_preference_options* options, int64_t pairs,
                                     const float* logp, const float* ref_logp,
                                     const int64_t* chosen, const int64_t* rejected, float* loss,
                                     float* score, float* logit, float* count, void* ws,
                                     size_t ws_bytes, void* hip_stream) {
  DORA_CHECK(check_batch(batch));
  DORA_CHECK(check_options(options));
  DORA_CHECK(check_pairs(pairs));
  const bool none = batch->tokens == 0, alone = pairs == 0, no_seq = batch->sequences == 0;
  DORA_CHECK(check_elem(logp, 4, none));
  DORA_CHECK(check_elem(ref_logp, 4, true));
  DORA_CHECK(check_elem(chosen, 8, alone));
  DORA_CHECK(check_elem(rejected, 8, alone));
  DORA_CHECK(check_elem(loss, 4, alone));
  DORA_CHECK(check_elem(logit, 4, alone));
  DORA_CHECK(check_elem(score, 4, no_seq));
  DORA_CHECK(check_elem(count, 4, no_seq));
  const Layout l = layout(*batch);
  DORA_CHECK(check_ws(ws, ws_bytes, l.bytes));
  const Batch b = device_batch(*batch);
  const Parts parts = parts_at(l, ws);
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  const Results to = {pairs, chosen, rejected, loss, score, logit, count};
  if (!none && b.tokens <= kSmallTokens && b.sequences + pairs <= kSmallRows) {
    if (no_seq && alone) return DORA_OK;
    const int64_t chunk = chunk_of(b.tokens, kSmall / 64);
    LaunchTimer timer("preference_small", st);
    auto kernel = ref_logp ? dora_preference_small<true> : dora_preference_small<false>;
    hipLaunchKernelGGL(kernel, dim3(1), dim3(kSmall), 0, st, b, parts, chunk, logp, ref_logp, numbers(*options),
                       to);
    HIP_TRY(hipGetLastError());
    return DORA_OK;
  }
  if (!none && !no_seq) {
    LaunchTimer timer("preference_sums", st);
    auto kernel = ref_logp ? dora_preference_sums<true> : dora_preference_sums<false>;
    hipLaunchKernelGGL(kernel, dim3(wave_grid(l.chunks)), dim3(kThreads), 0, st, b, parts, l.chunk,
                       logp, ref_logp);
    HIP_TRY(hipGetLastError());
  }
  if (no_seq && alone) return DORA_OK;
  LaunchTimer timer("preference_pairs", st);
  hipLaunchKernelGGL(dora_preference_pairs, dim3(wave_grid(b.sequences + pairs)), dim3(kThreads), 0,
                     st, b, parts, l.chunk, numbers(*options), to);
  HIP_TRY(hipGetLastError());
  return DORA_OK;
}

DORA_API int dora_preference_backward(const dora_token_batch* batch,
                                      const dora_preference_options* options, int64_t pairs,
                                      const float* grad_loss, const float* logit,
                                      const float* count, const int64_t* chosen,
                                      const int64_t* rejected, float* grad_logp, void* ws,
                                      size_t ws_bytes, void* hip_stream) {
  DORA_CHECK(check_batch(batch));
  DORA_CHECK(check_options(options));
  DORA_CHECK(check_pairs(pairs));
  const bool none = batch->tokens == 0, alone = pairs == 0, no_seq = batch->sequences == 0;
  DORA_CHECK(check_elem(grad_loss, 4, alone));
  DORA_CHECK(check_elem(logit, 4, alone));
  DORA_CHECK(check_elem(count, 4, no_seq || options->normalize == 0));
  DORA_CHECK(check_elem(chosen, 8, alone));
  DORA_CHECK(check_elem(rejected, 8, alone));
  DORA_CHECK(check_elem(grad_logp, 4, none));
  const Layout l = layout(*batch);
  DORA_CHECK(check_ws(ws, ws_bytes, l.bytes));
  if (none) return DORA_OK;
  const Batch b = device_batch(*batch);
  double* coef = reinterpret_cast<double*>(parts_at(l, ws).own);
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  const Pairs p = {numbers(*options), no_seq ? 0 : pairs, grad_loss, logit, count, chosen, rejected};
  const bool known = looks_first(b, p.count);
  if (known) {
    LaunchTimer timer("preference_coef", st);
    hipLaunchKernelGGL(dora_preference_coef, dim3(wave_grid(b.sequences)), dim3(kThreads), 0, st, b, p,
                       coef);
    HIP_TRY(hipGetLastError());
  }
  LaunchTimer timer("preference_grad", st);
  auto kernel = known ? dora_preference_grad<true> : dora_preference_grad<false>;
  // (waves of several rounds, as the sums': what a wave looks up counts for more tokens.  4.2M tokens
  // of 64 pairs 7.6 us, a round a wave 9.9)
  hipLaunchKernelGGL(kernel, dim3(wave_grid(l.chunks)), dim3(kThreads), 0, st, b, l.chunk, p, coef, grad_logp);
  HIP_TRY(hipGetLastError());
  return DORA_OK;
}

}  // extern "C"
