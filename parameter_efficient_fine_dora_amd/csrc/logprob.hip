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
// HIP holds the threads of a launch below 2^32: more rows than this share
// workgroups.
constexpr int64_t kMaxGrid = int64_t(1) << 23;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
// Beyond this |lse| the float32 lse itself is too coarse for exp(l - lse) (its
// half ulp is 3e-5 here), and the backward takes the row's maximum and sum anew.
constexpr float kCoarseLse = 1024.f;

// Whole numbers in the order of the floats: NaN above +inf, -0 equal to +0.
__device__ __forceinline__ uint32_t order_bits(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
// Larger value first, then the lower index.
__device__ __forceinline__ uint64_t order_key(float v, uint32_t index) {
  return ((uint64_t)order_bits(v) << 32) | (uint32_t)~index;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}

__device__ __forceinline__ float block_max(float v, float* lds) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v = fmaxf(v, lds[w]);
  return v;
}

__device__ __forceinline__ uint64_t block_max_key(uint64_t v, uint64_t* lds) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint64_t o = __shfl_xor((unsigned long long)v, off, 64);
    v = o > v ? o : v;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v = lds[w] > v ? lds[w] : v;
  return v;
}

// Maximum of a row of raw logits (NaN is passed over: it shows in the sums).
template <bool BF>
__device__ float row_max(const typename Elem<BF>::T* z, int64_t V, float* lds) {
  float m = kNegInf;
  for (int64_t j = (int64_t)threadIdx.x * Elem<BF>::kN; j < V; j += kThreads * Elem<BF>::kN) {
    float v[Elem<BF>::kN];
    load_part<BF>(z, j, V, kNegInf, v);
#pragma unroll
    for (int q = 0; q < Elem<BF>::kN; ++q) m = fmaxf(m, v[q]);
  }
  return block_max(m, lds);
}

// With e_j = exp(scale (z_j - m)): out[0] = sum e_j, out[1] = sum e_j scale (z_j - m).
// The differences are taken before scaling, so a row of the type's lowest
// values cannot overflow; -inf gives 0 in both sums.
template <bool BF>
__device__ void row_sums(const typename Elem<BF>::T* z, int64_t V, float m, float scale, float* out,
                         float* lds) {
  const float c2 = scale * kLog2e;
  float s = 0.f, u = 0.f;
  for (int64_t j = (int64_t)threadIdx.x * Elem<BF>::kN; j < V; j += kThreads * Elem<BF>::kN) {
    float v[Elem<BF>::kN];
    load_part<BF>(z, j, V, kNegInf, v);
#pragma unroll
    for (int q = 0; q < Elem<BF>::kN; ++q) {
      const float d = (v[q] - m) * c2;
      const float e = exp2f(d);
      s += e;
      u = fmaf(e, fmaxf(d, -200.f), u);
    }
  }
  out[0] = s;
  out[1] = u * kLn2;
  block_sum<kWaves, 2>(out, lds);
}

template <bool BF>
__global__ __launch_bounds__(kThreads) void dora_logprob_fwd(
    const void* logits, int64_t ld, const int64_t* targets, float* logp, float* entropy, float* lse,
    float* top_logp, int64_t* top_index, int64_t rows, int64_t V,
    int top, float scale) {
  using T = typename Elem<BF>::T;
  __shared__ float lds[4 * kWaves];
  __shared__ uint64_t lds_key[kWaves];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
  __syncthreads();   // the previous row's reductions have been read
  const T* z = reinterpret_cast<const T*>(logits) + row * ld;
  const int64_t y = targets[row];
  if (y < 0 || y >= V) {
    if (threadIdx.x == 0) {
      logp[row] = 0.f;
      if (entropy) entropy[row] = 0.f;
      if (lse) lse[row] = 0.f;
    }
    if ((int)threadIdx.x < top) {
      top_logp[row * top + threadIdx.x] = 0.f;
      top_index[row * top + threadIdx.x] = -1;
    }
    continue;
  }
  const float m = row_max<BF>(z, V, lds);
  const bool none = m == kNegInf;   // nothing left of the row (unless a NaN is in it)
  const float ref = none ? 0.f : m;
  float s[2];
  row_sums<BF>(z, V, ref, scale, s, lds + kWaves);
  const float log_s = logf(s[0]);
  const bool empty = none && s[0] == 0.f;
  if (threadIdx.x == 0) {
    const float at = (Elem<BF>::get(z + y) - ref) * scale;
    logp[row] = empty ? kNegInf : at - log_s;
    if (entropy) entropy[row] = empty ? 0.f : log_s - s[1] / s[0];
    if (lse) lse[row] = fmaf(ref, scale, log_s);
  }
  uint64_t last = ~uint64_t(0);
  for (int i = 0; i < top; ++i) {
    uint64_t best = 0;
    for (int64_t j = (int64_t)threadIdx.x * Elem<BF>::kN; j < V; j += kThreads * Elem<BF>::kN) {
      float v[Elem<BF>::kN];
      load_part<BF>(z, j, V, kNegInf, v);
#pragma unroll
      for (int q = 0; q < Elem<BF>::kN; ++q) {
        const uint64_t k = order_key(v[q], (uint32_t)(j + q));
        if (j + q < V && k < last && k > best) best = k;
      }
    }
    last = block_max_key(best, lds_key);
    if (threadIdx.x == 0) {
      const int64_t index = (uint32_t)~(uint32_t)last;
      top_index[row * top + i] = index;
      top_logp[row * top + i] =
          empty ? kNegInf : (Elem<BF>::get(z + index) - ref) * scale - log_s;
    }
  }
  }
}

template <bool BF>
__global__ __launch_bounds__(kThreads) void dora_logprob_bwd(
    const float* g_logp, const float* g_entropy, const void* logits, int64_t ld,
    const int64_t* targets, const float* lse, const float* entropy, void* grad, int64_t rows,
    int64_t V, float scale) {
  using E = Elem<BF>;
  using T = typename E::T;
  __shared__ float lds[3 * kWaves];
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
      const float m = row_max<BF>(z, V, lds);
      ref = m == kNegInf ? 0.f : m;
      float s[2];
      row_sums<BF>(z, V, ref, scale, s, lds + kWaves);
      zero = m == kNegInf && s[0] == 0.f;
      log_s = logf(s[0]);
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

bool shape_ok(const dora_logprob_shape& s) {
  return s.rows >= 0 && s.rows < kLimit && s.vocab >= 1 && s.vocab < kLimit && s.ld >= s.vocab &&
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

template <bool BF>
hipError_t forward(const dora_logprob_shape& s, const void* logits, const int64_t* targets,
                   float* logp, float* entropy, float* lse, float* top_logp, int64_t* top_index,
                   hipStream_t st) {
  LaunchTimer t("logprob_fwd", st);
  hipLaunchKernelGGL((dora_logprob_fwd<BF>), dim3((unsigned)std::min(s.rows, kMaxGrid)), dim3(kThreads),
                     0, st, logits, s.ld, targets, logp, entropy, lse, top_logp, top_index, s.rows, s.vocab, (int)s.top,
                     s.scale);
  return hipGetLastError();
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
  return 0;
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
              ? forward<true>(s, logits, targets, logp, entropy, lse, top_logp, top_index, st)
              : forward<false>(s, logits, targets, logp, entropy, lse, top_logp, top_index, st));
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
