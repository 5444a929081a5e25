// AdamW over many tensors in few launches, with states in float32 or in 8-bit
// codes; the gradients' global norm; and the 8-bit states' conversions.
//   g' = g factor,  m = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2
//   p = p (1 - lr decay) - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
// in float32, from the moments before their rounding; the parameter is rounded
// once (its master copy, if it has one, is float32).  Memory bounds all of it: a
// step moves 22 bytes an element for bf16 with float32 moments (28 with a master)
// and 10 with 8-bit moments.  151M bf16 with 8-bit moments: 239 us (6.4 TB/s), their
// values as bf16 75 us each (6.1 TB/s); 29M bf16 with masters: 140 us (5.9 TB/s),
// their norm 15 us and 5 us to add its parts.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/dora_finetune.h"
#include "checks.h"
#include "elem.h"
#include "kernels.h"
#include "launch_cut.h"

namespace dora {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 2048;                     // elements of a step's workgroup
constexpr int kVec = 8;                          // elements per thread where states have 8 bits
constexpr int kGroup = DORA_STATE_BLOCK / kVec;  // lanes that share an 8-bit block
static_assert(kGroup == 16, "an 8-bit block is one 16-lane row of a wave");
static_assert(kChunk % DORA_STATE_BLOCK == 0, "workgroups start at 8-bit blocks");

// The tensors of a launch travel in the kernel's arguments (under 4 KB, with as
// many tensors as fit), so a call needs no device table and no copy.  first[i]
// is the first workgroup of tensor i; workgroups past the last tensor do not
// exist.
struct StepNumbers {
  float beta1, beta2, c1, c2;   // c = 1 - beta
  float eps, decay, rest;       // decay + rest = 1 - lr weight_decay
  float step_size, inv_root;    // lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  const float* grad_scale;
  int count;
  int exact;                    // the root and the division in full (see update)
};
template <bool MASTER, bool S8>
struct StepArgs {
  static constexpr int kMax =
      (4096 - (int)sizeof(StepNumbers) - 8) / (8 * (5 + (S8 ? 2 : 0) + (MASTER ? 1 : 0)) + 4);
  StepNumbers h;
  int64_t n[kMax];
  void* param[kMax];
  const void* grad[kMax];
  void* exp_avg[kMax];
  void* exp_avg_sq[kMax];
  float* exp_avg_scale[S8 ? kMax : 1];
  float* exp_avg_sq_scale[S8 ? kMax : 1];
  float* master[MASTER ? kMax : 1];
  uint32_t first[kMax];
};
static_assert(sizeof(StepArgs<true, true>) <= 4096 && sizeof(StepArgs<true, false>) <= 4096 &&
                  sizeof(StepArgs<false, true>) <= 4096 && sizeof(StepArgs<false, false>) <= 4096,
              "kernel arguments");

constexpr int kNormChunk = 16384;   // elements of a workgroup of the norm, all loaded first
constexpr int kMaxGrads = 200;
struct NormArgs {
  const void* g[kMaxGrads];
  int64_t n[kMaxGrads];
  uint32_t first[kMaxGrads];
  int count;
};
static_assert(sizeof(NormArgs) <= 4096, "kernel arguments");

// The tensor that workgroup b belongs to, the last with first <= b: every lane
// compares some, one ballot counts.
__device__ __forceinline__ int tensor_of(const uint32_t* first, int count, uint32_t b) {
  int n = 0;
  for (int i = 0; i < count; i += 64) {
    const int k = i + (int)(threadIdx.x & 63);
    n += __popcll(__ballot(k < count && first[min(k, count - 1)] <= b));
  }
  return n - 1;
}

// A step touches every byte once and the next one comes a whole forward and
// backward later, so loads and stores go past the caches (37.8M float32
// elements with float32 states: 181 us against 201, 5.8 TB/s).  That asks for
// accesses that fill their lines: with float32 states a thread takes four
// elements (16 bytes of each such array), not eight.

// N elements (4 or 8) of an array from element i on, by 16-byte accesses (8 bytes
// for four bf16).  ALL: none is absent.
template <bool BF, int N, bool ALL>
__device__ __forceinline__ void load_n(const void* p, int64_t i, int64_t n, float* out) {
  using E = Elem<BF>;
  const typename E::T* q = reinterpret_cast<const typename E::T*>(p) + i;
  if (ALL || i + N <= n) {
    if constexpr (N >= E::kN) {
#pragma unroll
      for (int k = 0; k < N; k += E::kN) E::decode(E::raw_past(q + k), out + k);
    } else {
      typedef u32x2 Half __attribute__((aligned(2)));
      const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const Half*>(q));
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        out[2 * d] = bf_lo(v[d]);
        out[2 * d + 1] = bf_hi(v[d]);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) out[k] = i + k < n ? E::get(q + k) : 0.f;
  }
}
template <bool BF, int N, bool ALL>
__device__ __forceinline__ void store_n(void* p, int64_t i, int64_t n, const float* in) {
  using E = Elem<BF>;
  typename E::T* q = reinterpret_cast<typename E::T*>(p) + i;
  if (ALL || i + N <= n) {
    if constexpr (N >= E::kN) {
#pragma unroll
      for (int k = 0; k < N; k += E::kN) E::store_through(q + k, in + k);
    } else {
      typedef u32x2 Half __attribute__((aligned(2)));
      const u32x2 v = {pack_bf16x2(in[0], in[1]), pack_bf16x2(in[2], in[3])};
      __builtin_nontemporal_store(v, reinterpret_cast<Half*>(q));
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (i + k < n) E::put(q + k, in[k]);
  }
}

// Eight codes; absent ones are 0 and are not stored.
typedef u32x2 CodesRaw __attribute__((aligned(1)));
template <bool ALL>
__device__ __forceinline__ u32x2 load_codes(const void* p, int64_t i, int64_t n) {
  const uint8_t* q = reinterpret_cast<const uint8_t*>(p) + i;
  if (ALL || i + kVec <= n)
    return __builtin_nontemporal_load(reinterpret_cast<const CodesRaw*>(q));
  u32x2 v = {0u, 0u};
#pragma unroll
  for (int k = 0; k < kVec; ++k)
    if (i + k < n) v[k >> 2] |= (uint32_t)q[k] << (8 * (k & 3));
  return v;
}
template <bool ALL>
__device__ __forceinline__ void store_codes(void* p, int64_t i, int64_t n, u32x2 v) {
  uint8_t* q = reinterpret_cast<uint8_t*>(p) + i;
  if (ALL || i + kVec <= n) {
    __builtin_nontemporal_store(v, reinterpret_cast<CodesRaw*>(q));
    return;
  }
#pragma unroll
  for (int k = 0; k < kVec; ++k)
    if (i + k < n) q[k] = (uint8_t)(v[k >> 2] >> (8 * (k & 3)));
}

// Signed codes: value = scale c |c| / 127^2, read as c + 128 (one conversion
// from a byte).  Unsigned: scale (u / 255)^2.
constexpr uint32_t kFlip = 0x80808080u;
template <bool SIGNED>
__device__ __forceinline__ void decode8(u32x2 codes, float scale, float* out) {
  const float unit = scale * (SIGNED ? 1.f / (127.f * 127.f) : 1.f / (255.f * 255.f));
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    const uint32_t word = codes[k >> 2] ^ (SIGNED ? kFlip : 0u);
    const float byte = (float)((word >> (8 * (k & 3))) & 0xffu);
    const float c = SIGNED ? byte - 128.f : byte;
    out[k] = c * fabsf(c) * unit;
  }
}

// Largest magnitude of an 8-bit block, held by 16 lanes of 8; a NaN is kept.
__device__ __forceinline__ float maxnan(float a, float b) {
  return __builtin_elementwise_maximum(a, b);
}
__device__ __forceinline__ float block_scale(const float* v) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int k = 1; k < kVec; ++k) m = maxnan(m, fabsf(v[k]));
  m = maxnan(m, dpp_move<0xB1>(m));
  m = maxnan(m, dpp_move<0x4E>(m));
  m = maxnan(m, dpp_move<0x141>(m));
  return maxnan(m, dpp_move<0x140>(m));
}

// Codes of eight values, |c| = most sqrt(|v| / scale) rounded to nearest even by
// the conversion that puts a float into a byte (v_cvt_pk_u8_f32, which clamps to
// 0 .. 255; signed codes go through c + 128).  Reciprocal and root are the
// hardware's, 1 ulp each: far below the half step that rounding to a code costs.
// (With correctly rounded ones, here and in the step, as many codes differ from
// those of a plain float32 form, 3 or 4 in a million, and 151M elements with their
// moments' values take 514 us against 393.)
// Scales outside their range are divided by.  A block whose scale is not finite
// keeps that scale and codes of 0: its values read back as NaN.
template <bool SIGNED>
__device__ __forceinline__ u32x2 encode8(const float* v, float scale) {
  constexpr float most = SIGNED ? 127.f : 255.f;
  const bool usual = scale > 0x1p-100f && scale < 0x1p100f;
  const float inv = usual ? __builtin_amdgcn_rcpf(scale) : 0.f;
  u32x2 codes = {0u, 0u};
  auto put = [&](int k, float root) {
    float f;
    if (SIGNED)
      f = fmaf(most, copysignf(root, v[k]), 128.f);
    else   // a nonzero value keeps code 1
      f = fmaxf(most * root, __builtin_amdgcn_fmed3f(v[k] * 3e38f, 0.f, 1.f));
    codes[k >> 2] = __builtin_amdgcn_cvt_pk_u8_f32(f, k & 3, codes[k >> 2]);
  };
#pragma unroll
  for (int k = 0; k < kVec; ++k) put(k, __builtin_amdgcn_sqrtf(fabsf(v[k]) * inv));
  if (SIGNED) codes ^= kFlip;
  if (!usual) {
    codes = u32x2{0u, 0u};
    if (scale > 0.f && scale < __builtin_huge_valf()) {
#pragma unroll
      for (int k = 0; k < kVec; ++k) put(k, sqrtf(fabsf(v[k]) / scale));
      if (SIGNED) codes ^= kFlip;
    }
  }
  return codes;
}

// ---- the step -------------------------------------------------------------------
// N elements: the moments, their root (into r) and the parameter.  The root and
// the reciprocal of the denominator are the hardware's (1 ulp each), which take a
// second moment under 2^-126 for 0; where eps does not cover that (see the host's
// choice of `exact`), both are correctly rounded.  What rounding the
// decay's factor leaves is added with the update, and the sum with the decayed
// parameter is rounded once: as a float32 factor alone, a decay of 1e-7 is 19% off
// and one of 1e-8 none at all.
template <int N>
__device__ __forceinline__ void update(const StepNumbers& h, float gs, const float* g, float* p,
                                       float* m, float* v, float* r) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float gk = g[k] * gs;
    m[k] = fmaf(h.beta1, m[k], h.c1 * gk);
    v[k] = fmaf(h.beta2, v[k], h.c2 * gk * gk);
  }
  float q[N];
  if (h.exact) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      r[k] = sqrtf(v[k]);
      q[k] = m[k] / fmaf(r[k], h.inv_root, h.eps);
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      r[k] = __builtin_amdgcn_sqrtf(v[k]);
      q[k] = m[k] * __builtin_amdgcn_rcpf(fmaf(r[k], h.inv_root, h.eps));
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float change = -h.step_size * q[k];
    if (h.rest != 0.f) change = fmaf(p[k], h.rest, change);
    p[k] = fmaf(p[k], h.decay, change);
  }
}

template <bool PBF, bool GBF, bool MASTER, bool S8>
__global__ __launch_bounds__(kChunk / (S8 ? 8 : 4)) void dora_adamw_kernel(
    const StepArgs<MASTER, S8> a) {
  constexpr int N = S8 ? kVec : 4;
  const int t = __builtin_amdgcn_readfirstlane(tensor_of(a.first, a.h.count, blockIdx.x));
  const int64_t n = a.n[t];
  const int64_t start = (int64_t)(blockIdx.x - a.first[t]) * kChunk;
  const int64_t i = start + threadIdx.x * N;
  const float gs = a.h.grad_scale ? *a.h.grad_scale : 1.f;
  void* weight = MASTER ? (void*)a.master[t] : a.param[t];
  auto step = [&](auto all) {
    constexpr bool ALL = decltype(all)::value;
    float p[N], g[N], m[N], v[N], r[N];
    load_n<PBF && !MASTER, N, ALL>(weight, i, n, p);
    load_n<GBF, N, ALL>(a.grad[t], i, n, g);
    if constexpr (S8) {
      const int64_t block = i / DORA_STATE_BLOCK;
      const u32x2 mc = load_codes<ALL>(a.exp_avg[t], i, n);
      const u32x2 vc = load_codes<ALL>(a.exp_avg_sq[t], i, n);
      decode8<true>(mc, a.exp_avg_scale[t][block], m);
      decode8<false>(vc, a.exp_avg_sq_scale[t][block], v);
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] *= v[k];
    } else {
      load_n<false, N, ALL>(a.exp_avg[t], i, n, m);
      load_n<false, N, ALL>(a.exp_avg_sq[t], i, n, v);
    }
    update<N>(a.h, gs, g, p, m, v, r);
    if (MASTER) store_n<false, N, ALL>(weight, i, n, p);
    store_n<PBF, N, ALL>(a.param[t], i, n, p);
    if constexpr (S8) {
      const int64_t block = i / DORA_STATE_BLOCK;
      const float ms = block_scale(m), vs = block_scale(r);
      store_codes<ALL>(a.exp_avg[t], i, n, encode8<true>(m, ms));
      store_codes<ALL>(a.exp_avg_sq[t], i, n, encode8<false>(r, vs));
      if ((threadIdx.x & (kGroup - 1)) == 0) {
        a.exp_avg_scale[t][block] = ms;
        a.exp_avg_sq_scale[t][block] = vs;
      }
    } else {
      store_n<false, N, ALL>(a.exp_avg[t], i, n, m);
      store_n<false, N, ALL>(a.exp_avg_sq[t], i, n, v);
    }
  };
  if (start + kChunk <= n) {
    step(std::true_type());
  } else {
    // an 8-bit block's 16 lanes stay together: those past the end carry zeros
    const int64_t last = S8 ? (n + DORA_STATE_BLOCK - 1) / DORA_STATE_BLOCK * DORA_STATE_BLOCK : n;
    if (i < last) step(std::false_type());
  }
}

// ---- the gradients' norm ------------------------------------------------------------
__device__ __forceinline__ double block_sum_f64(double v, double* lds) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
  for (unsigned w = 1; w < blockDim.x / 64; ++w) v += lds[w];
  return v;
}

// One workgroup's elements, squared and summed in float64 (a float32 square
// passes the type's range from 1.8e19 on).
template <bool GBF>
__global__ __launch_bounds__(kThreads) void dora_grad_norm_parts(const NormArgs a, double* part) {
  __shared__ double lds[kThreads / 64];
  using E = Elem<GBF>;
  using T = typename E::T;
  const int t = __builtin_amdgcn_readfirstlane(tensor_of(a.first, a.count, blockIdx.x));
  const int64_t n = a.n[t];
  const int64_t start = (int64_t)(blockIdx.x - a.first[t]) * kNormChunk;
  const T* g = reinterpret_cast<const T*>(a.g[t]) + start;
  double sum = 0.0;
  constexpr int kLoads = kNormChunk / kThreads / E::kN;
  if (start + kNormChunk <= n) {
    typename E::Vec raw[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) raw[u] = E::raw(g + (u * kThreads + threadIdx.x) * E::kN);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      float v[E::kN];
      E::decode(raw[u], v);
#pragma unroll
      for (int k = 0; k < E::kN; ++k) sum = fma((double)v[k], (double)v[k], sum);
    }
  } else {
    for (int64_t i = threadIdx.x * E::kN; i < n - start; i += kThreads * E::kN) {
      float v[E::kN];
      load_part<GBF>(g, i, n - start, 0.f, v);
#pragma unroll
      for (int k = 0; k < E::kN; ++k) sum = fma((double)v[k], (double)v[k], sum);
    }
  }
  sum = block_sum_f64(sum, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ __launch_bounds__(1024) void dora_grad_norm_finish(const double* part, int64_t parts,
                                                              double max_norm, float* norm,
                                                              float* scale) {
  __shared__ double lds[16];
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < parts; i += 1024) sum += part[i];
  sum = block_sum_f64(sum, lds);
  if (threadIdx.x == 0) {
    const double v = sqrt(sum);
    *norm = (float)v;
    // a NaN norm gives a NaN factor
    const double f = max_norm / (v + 1e-6);
    if (scale) *scale = f > 1.0 ? 1.f : (float)f;
  }
}

// ---- 8-bit states and their values ----------------------------------------------------
template <bool BF, bool SECOND>
__global__ __launch_bounds__(kThreads) void dora_state_values(const void* codes,
                                                              const float* scales, void* out,
                                                              int64_t n) {
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kVec;
  if (i >= n) return;
  float v[kVec];
  decode8<!SECOND>(load_codes<false>(codes, i, n), scales[i / DORA_STATE_BLOCK], v);
#pragma unroll
  for (int k = 0; k < kVec; ++k)
    if (SECOND) v[k] *= v[k];
  store_n<BF, kVec, false>(out, i, n, v);
}

template <bool SECOND>
__global__ __launch_bounds__(kThreads) void dora_state_codes(const float* values, void* codes,
                                                             float* scales, int64_t n) {
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kVec;
  const int64_t block = i / DORA_STATE_BLOCK;
  if (block * DORA_STATE_BLOCK >= n) return;
  float v[kVec];
  load_n<false, kVec, false>(values, i, n, v);
#pragma unroll
  for (int k = 0; k < kVec; ++k)
    if (SECOND) v[k] = sqrtf(v[k]);
  const float s = block_scale(v);
  store_codes<false>(codes, i, n, encode8<!SECOND>(v, s));
  if ((threadIdx.x & (kGroup - 1)) == 0) scales[block] = s;
}

// ---- host -----------------------------------------------------------------------
constexpr int64_t kMaxElems = int64_t(1) << 34;

int64_t norm_chunks(int64_t n) { return (n + kNormChunk - 1) / kNormChunk; }
bool dtype_ok(int dt) { return dt == DORA_F32 || dt == DORA_BF16; }
size_t esize(int dt) { return dt == DORA_BF16 ? 2 : 4; }

int check_tensors(const dora_adamw_tensor* t, int64_t count) {
  if (count < 0 || count >= kMaxElems) return DORA_ERR_SHAPE;
  if (count > 0 && !t) return DORA_ERR_NULL;
  for (int64_t i = 0; i < count; ++i)
    if (t[i].n < 0 || t[i].n >= kMaxElems) return DORA_ERR_SHAPE;
  return DORA_OK;
}

template <bool PBF, bool GBF, bool MASTER, bool S8>
hipError_t run_step(const dora_adamw_tensor* tensors, int64_t count, const StepNumbers& h,
                    hipStream_t st) {
  using Args = StepArgs<MASTER, S8>;
  constexpr int threads = kChunk / (S8 ? 8 : 4);
  Args a;
  a.h = h;
  // the byte that element `at` of an array of so many bytes an element starts at
  auto from = [](auto* p, int64_t at, int bytes) {
    using P = decltype(p);
    return reinterpret_cast<P>((uintptr_t)p + (uintptr_t)at * bytes);
  };
  return cut_launches<hipError_t>(
      count, kChunk, Args::kMax, launch_blocks(threads), [&](int64_t i) { return tensors[i].n; },
      [&](int k, int64_t i, int64_t at, int64_t n, int64_t block) {
        const dora_adamw_tensor& t = tensors[i];
        a.n[k] = n;
        a.param[k] = from(t.param, at, PBF ? 2 : 4);
        a.grad[k] = from(t.grad, at, GBF ? 2 : 4);
        a.exp_avg[k] = from(t.exp_avg, at, S8 ? 1 : 4);
        a.exp_avg_sq[k] = from(t.exp_avg_sq, at, S8 ? 1 : 4);
        if (S8) {   // pieces start at 8-bit blocks
          a.exp_avg_scale[k] = t.exp_avg_scale + at / DORA_STATE_BLOCK;
          a.exp_avg_sq_scale[k] = t.exp_avg_sq_scale + at / DORA_STATE_BLOCK;
        }
        if (MASTER) a.master[k] = t.master + at;
        a.first[k] = (uint32_t)block;
      },
      [&](int pieces, int64_t blocks) {
        a.h.count = pieces;
        LaunchTimer timer("adamw", st);
        hipLaunchKernelGGL((dora_adamw_kernel<PBF, GBF, MASTER, S8>), dim3((unsigned)blocks),
                           dim3(threads), 0, st, a);
        return hipGetLastError();
      });
}

// The step for the types of a call: a float32 parameter is its own master.
hipError_t step_for(const dora_adamw_tensor* t, int64_t n, const dora_adamw_options& o, bool master,
                    const StepNumbers& h, hipStream_t st) {
  const bool gbf = o.grad_dtype == DORA_BF16, s8 = o.state_bits == 8;
  auto pick = [&](auto pbf, auto mst) {
    constexpr bool P = decltype(pbf)::value, M = decltype(mst)::value;
    if (s8) return gbf ? run_step<P, true, M, true>(t, n, h, st) : run_step<P, false, M, true>(t, n, h, st);
    return gbf ? run_step<P, true, M, false>(t, n, h, st) : run_step<P, false, M, false>(t, n, h, st);
  };
  if (o.param_dtype == DORA_F32) return pick(std::false_type(), std::false_type());
  return master ? pick(std::true_type(), std::true_type()) : pick(std::true_type(), std::false_type());
}

bool options_ok(const dora_adamw_options& o) {
  return o.reserved == 0 && (o.state_bits == 32 || o.state_bits == 8) && std::isfinite(o.lr) &&
         std::isfinite(o.weight_decay) && std::isfinite(o.eps) && o.eps >= 0 && o.beta1 >= 0 &&
         o.beta1 < 1 && o.beta2 >= 0 && o.beta2 < 1 && o.step >= 1;
}

static_assert(kMaxElems / (kThreads * kVec) <= launch_blocks(kThreads),
              "the conversions' elements fit one launch");

}  // namespace
}  // namespace dora

using namespace dora;

extern "C" {

DORA_API int dora_adamw_step(const dora_adamw_tensor* tensors, int64_t count,
                             const dora_adamw_options* options, void* hip_stream) {
  if (!options) return DORA_ERR_NULL;
  const dora_adamw_options& o = *options;
  if (!dtype_ok(o.param_dtype) || !dtype_ok(o.grad_dtype)) return DORA_ERR_DTYPE;
  if (!options_ok(o)) return DORA_ERR_FLAGS;
  DORA_CHECK(check_tensors(tensors, count));
  DORA_CHECK(check_elem(o.grad_scale, 4, true));
  bool master = false;
  bool any = false;
  for (int64_t i = 0; i < count; ++i) {
    const dora_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    if (!any) master = t.master != nullptr;
    any = true;
    if ((t.master != nullptr) != master) return DORA_ERR_NULL;
    DORA_CHECK(check_elem(t.param, esize(o.param_dtype), false));
    DORA_CHECK(check_elem(t.grad, esize(o.grad_dtype), false));
    DORA_CHECK(check_elem(t.exp_avg, o.state_bits == 8 ? 1 : 4, false));
    DORA_CHECK(check_elem(t.exp_avg_sq, o.state_bits == 8 ? 1 : 4, false));
    DORA_CHECK(check_elem(t.exp_avg_scale, 4, o.state_bits == 32));
    DORA_CHECK(check_elem(t.exp_avg_sq_scale, 4, o.state_bits == 32));
    DORA_CHECK(check_elem(t.master, 4, true));
  }
  if (master && o.param_dtype != DORA_BF16) return DORA_ERR_DTYPE;
  StepNumbers h;
  h.beta1 = (float)o.beta1;
  h.beta2 = (float)o.beta2;
  h.c1 = (float)(1.0 - o.beta1);
  h.c2 = (float)(1.0 - o.beta2);
  h.eps = (float)o.eps;
  const double decay = o.lr * o.weight_decay;
  h.decay = (float)(1.0 - decay);
  // under 2^-15 of the decay (always where that is 2^-10 or more) the rest is left out
  h.rest = (float)(1.0 - decay - (double)h.decay);
  if (std::fabs(h.rest) <= 0x1p-15 * std::fabs(decay)) h.rest = 0.f;
  h.step_size = (float)(o.lr / (1.0 - std::pow(o.beta1, (double)o.step)));
  h.inv_root = (float)(1.0 / std::sqrt(1.0 - std::pow(o.beta2, (double)o.step)));
  // a lost root is under 2^-63: with its correction 2^-24 of this eps at most
  h.exact = o.eps < 0x1p-39 * (double)h.inv_root;
  h.grad_scale = o.grad_scale;
  h.count = 0;
  HIP_TRY(step_for(tensors, count, o, master, h, reinterpret_cast<hipStream_t>(hip_stream)));
  return DORA_OK;
}

DORA_API size_t dora_grad_norm_workspace_bytes(const dora_adamw_tensor* tensors, int64_t count) {
  if (check_tensors(tensors, count) != DORA_OK) return 0;
  int64_t parts = 0;
  for (int64_t i = 0; i < count; ++i) parts += norm_chunks(tensors[i].n);
  return (size_t)parts * sizeof(double);
}

DORA_API int dora_grad_norm(const dora_adamw_tensor* tensors, int64_t count, int32_t grad_dtype,
                            double max_norm, float* norm, float* scale, void* ws, size_t ws_bytes,
                            void* hip_stream) {
  if (!dtype_ok(grad_dtype)) return DORA_ERR_DTYPE;
  if (!std::isfinite(max_norm) || max_norm < 0) return DORA_ERR_FLAGS;
  DORA_CHECK(check_tensors(tensors, count));
  DORA_CHECK(check_elem(norm, 4, false));
  DORA_CHECK(check_elem(scale, 4, true));
  for (int64_t i = 0; i < count; ++i)
    DORA_CHECK(check_elem(tensors[i].grad, esize(grad_dtype), tensors[i].n == 0));
  DORA_CHECK(check_ws(ws, ws_bytes, dora_grad_norm_workspace_bytes(tensors, count)));
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  double* part = reinterpret_cast<double*>(ws);
  int64_t done = 0;
  NormArgs a;
  HIP_TRY(cut_launches<hipError_t>(
      count, kNormChunk, kMaxGrads, launch_blocks(kThreads),
      [&](int64_t i) { return tensors[i].n; },
      [&](int k, int64_t i, int64_t at, int64_t n, int64_t block) {
        a.g[k] = reinterpret_cast<const uint8_t*>(tensors[i].grad) + at * esize(grad_dtype);
        a.n[k] = n;
        a.first[k] = (uint32_t)block;
      },
      [&](int pieces, int64_t blocks) {
        a.count = pieces;
        LaunchTimer timer("grad_norm", st);
        if (grad_dtype == DORA_BF16)
          hipLaunchKernelGGL((dora_grad_norm_parts<true>), dim3((unsigned)blocks), dim3(kThreads), 0,
                             st, a, part + done);
        else
          hipLaunchKernelGGL((dora_grad_norm_parts<false>), dim3((unsigned)blocks), dim3(kThreads), 0,
                             st, a, part + done);
        done += blocks;
        return hipGetLastError();
      }));
  LaunchTimer timer("grad_norm_finish", st);
  hipLaunchKernelGGL(dora_grad_norm_finish, dim3(1), dim3(1024), 0, st, part, done, max_norm, norm,
                     scale);
  HIP_TRY(hipGetLastError());
  return DORA_OK;
}

DORA_API int dora_adamw_dequantize(const void* codes, const float* scales, int64_t n,
                                   int second_moment, void* out, int32_t out_dtype,
                                   void* hip_stream) {
  if (!dtype_ok(out_dtype)) return DORA_ERR_DTYPE;
  if (n < 0 || n >= kMaxElems) return DORA_ERR_SHAPE;
  DORA_CHECK(check_elem(codes, 1, n == 0));
  DORA_CHECK(check_elem(scales, 4, n == 0));
  DORA_CHECK(check_elem(out, esize(out_dtype), n == 0));
  if (n == 0) return DORA_OK;
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  const dim3 grid((unsigned)((n + kThreads * kVec - 1) / (kThreads * kVec))), block(kThreads);
  LaunchTimer timer("state_values", st);
  if (out_dtype == DORA_BF16) {
    if (second_moment)
      hipLaunchKernelGGL((dora_state_values<true, true>), grid, block, 0, st, codes, scales, out, n);
    else
      hipLaunchKernelGGL((dora_state_values<true, false>), grid, block, 0, st, codes, scales, out,
                         n);
  } else {
    if (second_moment)
      hipLaunchKernelGGL((dora_state_values<false, true>), grid, block, 0, st, codes, scales, out,
                         n);
    else
      hipLaunchKernelGGL((dora_state_values<false, false>), grid, block, 0, st, codes, scales, out,
                         n);
  }
  HIP_TRY(hipGetLastError());
  return DORA_OK;
}

DORA_API int dora_adamw_quantize(const float* values, int64_t n, int second_moment, void* codes,
                                 float* scales, void* hip_stream) {
  if (n < 0 || n >= kMaxElems) return DORA_ERR_SHAPE;
  DORA_CHECK(check_elem(values, 4, n == 0));
  DORA_CHECK(check_elem(codes, 1, n == 0));
  DORA_CHECK(check_elem(scales, 4, n == 0));
  if (n == 0) return DORA_OK;
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  const dim3 grid((unsigned)((n + kThreads * kVec - 1) / (kThreads * kVec))), block(kThreads);
  LaunchTimer timer("state_codes", st);
  if (second_moment)
    hipLaunchKernelGGL((dora_state_codes<true>), grid, block, 0, st, values, codes, scales, n);
  else
    hipLaunchKernelGGL((dora_state_codes<false>), grid, block, 0, st, values, codes, scales, n);
  HIP_TRY(hipGetLastError());
  return DORA_OK;
}

}  // extern "C"
