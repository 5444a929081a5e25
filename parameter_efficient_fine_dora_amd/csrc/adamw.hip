// AdamW over many tensors in few launches, with states in float32 or in 8-bit
// codes; the gradients' global norm; and the 8-bit states' conversions.
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
constexpr int kVec = 8;                          // elements per thread and step
constexpr int kChunk = kThreads * kVec * 2;      // elements per workgroup
constexpr int kGroup = DORA_STATE_BLOCK / kVec;  // lanes that share an 8-bit block
static_assert(kGroup == 16, "an 8-bit block is one 16-lane row of a wave");
static_assert(kChunk % DORA_STATE_BLOCK == 0, "workgroups start at 8-bit blocks");

// The tensors of a launch travel in the kernel's arguments (under 4 KB), so a
// call needs no device table and no copy.  first[i] is the first workgroup of
// tensor i; workgroups past the last tensor do not exist.
constexpr int kMaxTensors = 54;
struct StepArgs {
  dora_adamw_tensor t[kMaxTensors];
  uint32_t first[kMaxTensors];
  int count;
  float beta1, beta2, c1, c2;   // c = 1 - beta
  float eps, decay;             // decay = 1 - lr weight_decay
  float step_size, inv_root;    // lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  const float* grad_scale;
};
static_assert(sizeof(StepArgs) <= 4096, "kernel arguments");

constexpr int kMaxGrads = 160;
struct NormArgs {
  const void* g[kMaxGrads];
  int64_t n[kMaxGrads];
  uint32_t first[kMaxGrads];
  int count;
};
static_assert(sizeof(NormArgs) <= 4096, "kernel arguments");

// Index of the tensor that workgroup b belongs to: the last with first <= b.
__device__ __forceinline__ int tensor_of(const uint32_t* first, int count, uint32_t b) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= b)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

template <bool BF>
__device__ __forceinline__ void load8(const void* p, int64_t i, int64_t n, float* out) {
  const typename Elem<BF>::T* q = reinterpret_cast<const typename Elem<BF>::T*>(p);
#pragma unroll
  for (int k = 0; k < kVec; k += Elem<BF>::kN) load_part<BF>(q, i + k, n, 0.f, out + k);
}
template <bool BF>
__device__ __forceinline__ void store8(void* p, int64_t i, int64_t n, const float* in) {
  typename Elem<BF>::T* q = reinterpret_cast<typename Elem<BF>::T*>(p);
#pragma unroll
  for (int k = 0; k < kVec; k += Elem<BF>::kN) store_part<BF>(q, i + k, n, in + k);
}

// Eight codes; absent ones are 0 and are not stored.
typedef u32x2 CodesRaw __attribute__((aligned(1)));
__device__ __forceinline__ u32x2 load_codes(const void* p, int64_t i, int64_t n) {
  const uint8_t* q = reinterpret_cast<const uint8_t*>(p) + i;
  if (i + kVec <= n) return *reinterpret_cast<const CodesRaw*>(q);
  u32x2 v = {0u, 0u};
#pragma unroll
  for (int k = 0; k < kVec; ++k)
    if (i + k < n) v[k >> 2] |= (uint32_t)q[k] << (8 * (k & 3));
  return v;
}
__device__ __forceinline__ void store_codes(void* p, int64_t i, int64_t n, u32x2 v) {
  uint8_t* q = reinterpret_cast<uint8_t*>(p) + i;
  if (i + kVec <= n) {
    *reinterpret_cast<CodesRaw*>(q) = v;
    return;
  }
#pragma unroll
  for (int k = 0; k < kVec; ++k)
    if (i + k < n) q[k] = (uint8_t)(v[k >> 2] >> (8 * (k & 3)));
}

// Signed codes: value = scale c |c| / 127^2.  Unsigned: scale (u / 255)^2.
template <bool SIGNED>
__device__ __forceinline__ void decode8(u32x2 codes, float scale, float* out) {
  const float unit = scale * (SIGNED ? 1.f / (127.f * 127.f) : 1.f / (255.f * 255.f));
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    const uint32_t byte = (codes[k >> 2] >> (8 * (k & 3))) & 0xffu;
    const float c = SIGNED ? (float)(int8_t)byte : (float)byte;
    out[k] = SIGNED ? c * fabsf(c) * unit : c * c * unit;
  }
}

// Largest magnitude of an 8-bit block, held by 16 lanes of 8.  Compared as
// whole numbers: a NaN is above every number and is kept.
__device__ __forceinline__ float block_scale(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < kVec; ++k) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
#pragma unroll
  for (int off = kGroup / 2; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
  return __uint_as_float(m);
}

// Codes of eight values, |c| = round(most sqrt(|v| / scale)).  A block whose
// scale is not finite keeps that scale and codes of 0: all its values read back
// as NaN.
template <bool SIGNED>
__device__ __forceinline__ u32x2 encode8(const float* v, float scale) {
  const float most = SIGNED ? 127.f : 255.f;
  const bool ok = scale > 0.f && scale < __builtin_huge_valf();
  // the smallest scales have no finite reciprocal
  const float inv = 1.f / scale;
  const bool tiny = !(inv < __builtin_huge_valf());
  u32x2 codes = {0u, 0u};
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    const float share = tiny ? fabsf(v[k]) / scale : fabsf(v[k]) * inv;
    float c = rintf(most * sqrtf(share));
    c = fminf(c, most);
    if (!SIGNED && v[k] > 0.f) c = fmaxf(c, 1.f);
    int code = ok ? (int)c : 0;
    if (SIGNED && v[k] < 0.f) code = -code;
    codes[k >> 2] |= ((uint32_t)code & 0xffu) << (8 * (k & 3));
  }
  return codes;
}

// ---- the step -------------------------------------------------------------------
template <bool PBF, bool GBF, bool MASTER, bool S8>
__global__ __launch_bounds__(kThreads) void dora_adamw_kernel(const StepArgs a) {
  const int ti = tensor_of(a.first, a.count, blockIdx.x);
  const dora_adamw_tensor& t = a.t[ti];
  const int64_t n = t.n;
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const int64_t base = (int64_t)(blockIdx.x - a.first[ti]) * kChunk + threadIdx.x * kVec;
  for (int64_t i = base; i < base + kChunk; i += kThreads * kVec) {
    // an 8-bit block's 16 lanes stay together: those past the end carry zeros
    const int64_t block = i / DORA_STATE_BLOCK;
    if (i >= n && (!S8 || block * DORA_STATE_BLOCK >= n)) break;
    float p[kVec], g[kVec], m[kVec], v[kVec], r[kVec];
    if (MASTER)
      load8<false>(t.master, i, n, p);
    else
      load8<PBF>(t.param, i, n, p);
    load8<GBF>(t.grad, i, n, g);
    if (S8) {
      decode8<true>(load_codes(t.exp_avg, i, n), t.exp_avg_scale[block], m);
      decode8<false>(load_codes(t.exp_avg_sq, i, n), t.exp_avg_sq_scale[block], r);
#pragma unroll
      for (int k = 0; k < kVec; ++k) v[k] = r[k] * r[k];
    } else {
      load8<false>(t.exp_avg, i, n, m);
      load8<false>(t.exp_avg_sq, i, n, v);
    }
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const float gk = g[k] * gs;
      m[k] = fmaf(a.beta1, m[k], a.c1 * gk);
      v[k] = fmaf(a.beta2, v[k], a.c2 * gk * gk);
      r[k] = sqrtf(v[k]);
      p[k] = fmaf(-a.step_size, m[k] / fmaf(r[k], a.inv_root, a.eps), p[k] * a.decay);
    }
    if (MASTER) store8<false>(t.master, i, n, p);
    store8<PBF>(t.param, i, n, p);
    if (S8) {
      const float ms = block_scale(m), rs = block_scale(r);
      store_codes(t.exp_avg, i, n, encode8<true>(m, ms));
      store_codes(t.exp_avg_sq, i, n, encode8<false>(r, rs));
      if ((threadIdx.x & (kGroup - 1)) == 0) {
        t.exp_avg_scale[block] = ms;
        t.exp_avg_sq_scale[block] = rs;
      }
    } else {
      store8<false>(t.exp_avg, i, n, m);
      store8<false>(t.exp_avg_sq, i, n, v);
    }
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

template <bool GBF>
__global__ __launch_bounds__(kThreads) void dora_grad_norm_parts(const NormArgs a, double* part) {
  __shared__ double lds[kThreads / 64];
  const int ti = tensor_of(a.first, a.count, blockIdx.x);
  const int64_t n = a.n[ti];
  const int64_t base = (int64_t)(blockIdx.x - a.first[ti]) * kChunk + threadIdx.x * kVec;
  double sum = 0.0;
  for (int64_t i = base; i < base + kChunk && i < n; i += kThreads * kVec) {
    float g[kVec];
    load8<GBF>(a.g[ti], i, n, g);
#pragma unroll
    for (int k = 0; k < kVec; ++k) sum = fma((double)g[k], (double)g[k], sum);
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
  decode8<!SECOND>(load_codes(codes, i, n), scales[i / DORA_STATE_BLOCK], v);
#pragma unroll
  for (int k = 0; k < kVec; ++k)
    if (SECOND) v[k] *= v[k];
  store8<BF>(out, i, n, v);
}

template <bool SECOND>
__global__ __launch_bounds__(kThreads) void dora_state_codes(const float* values, void* codes,
                                                             float* scales, int64_t n) {
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kVec;
  const int64_t block = i / DORA_STATE_BLOCK;
  if (block * DORA_STATE_BLOCK >= n) return;
  float v[kVec];
  load8<false>(values, i, n, v);
#pragma unroll
  for (int k = 0; k < kVec; ++k)
    if (SECOND) v[k] = sqrtf(v[k]);
  const float s = block_scale(v);
  store_codes(codes, i, n, encode8<!SECOND>(v, s));
  if ((threadIdx.x & (kGroup - 1)) == 0) scales[block] = s;
}

// ---- host -----------------------------------------------------------------------
constexpr int64_t kMaxElems = int64_t(1) << 34;

int64_t chunks(int64_t n) { return (n + kChunk - 1) / kChunk; }
bool dtype_ok(int dt) { return dt == DORA_F32 || dt == DORA_BF16; }
size_t esize(int dt) { return dt == DORA_BF16 ? 2 : 4; }

int check_tensors(const dora_adamw_tensor* t, int64_t count) {
  if (count < 0 || count >= kMaxElems) return DORA_ERR_SHAPE;
  if (count > 0 && !t) return DORA_ERR_NULL;
  for (int64_t i = 0; i < count; ++i)
    if (t[i].n < 0 || t[i].n >= kMaxElems) return DORA_ERR_SHAPE;
  return DORA_OK;
}

// HIP holds the threads of a launch below 2^32: a call's tensors are cut into
// runs of at most this many workgroups.
constexpr int64_t kMaxGrid = int64_t(1) << 23;

template <bool PBF, bool GBF, bool MASTER>
void launch_step(const StepArgs& a, unsigned blocks, int bits, hipStream_t st) {
  if (bits == 8)
    hipLaunchKernelGGL((dora_adamw_kernel<PBF, GBF, MASTER, true>), dim3(blocks), dim3(kThreads), 0,
                       st, a);
  else
    hipLaunchKernelGGL((dora_adamw_kernel<PBF, GBF, MASTER, false>), dim3(blocks), dim3(kThreads),
                       0, st, a);
}

hipError_t run_step(const StepArgs& a, int64_t blocks, const dora_adamw_options& o, bool master,
                    hipStream_t st) {
  LaunchTimer timer("adamw", st);
  const unsigned b = (unsigned)blocks;
  const bool gbf = o.grad_dtype == DORA_BF16;
  if (o.param_dtype == DORA_F32)
    gbf ? launch_step<false, true, false>(a, b, o.state_bits, st)
        : launch_step<false, false, false>(a, b, o.state_bits, st);
  else if (master)
    gbf ? launch_step<true, true, true>(a, b, o.state_bits, st)
        : launch_step<true, false, true>(a, b, o.state_bits, st);
  else
    gbf ? launch_step<true, true, false>(a, b, o.state_bits, st)
        : launch_step<true, false, false>(a, b, o.state_bits, st);
  return hipGetLastError();
}

bool options_ok(const dora_adamw_options& o) {
  return o.reserved == 0 && (o.state_bits == 32 || o.state_bits == 8) && std::isfinite(o.lr) &&
         std::isfinite(o.weight_decay) && std::isfinite(o.eps) && o.eps >= 0 && o.beta1 >= 0 &&
         o.beta1 < 1 && o.beta2 >= 0 && o.beta2 < 1 && o.step >= 1;
}

static_assert(kMaxElems / kChunk <= kMaxGrid, "one tensor fits one launch");

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
  StepArgs a;
  a.beta1 = (float)o.beta1;
  a.beta2 = (float)o.beta2;
  a.c1 = (float)(1.0 - o.beta1);
  a.c2 = (float)(1.0 - o.beta2);
  a.eps = (float)o.eps;
  a.decay = (float)(1.0 - o.lr * o.weight_decay);
  a.step_size = (float)(o.lr / (1.0 - std::pow(o.beta1, (double)o.step)));
  a.inv_root = (float)(1.0 / std::sqrt(1.0 - std::pow(o.beta2, (double)o.step)));
  a.grad_scale = o.grad_scale;
  a.count = 0;
  int64_t blocks = 0;
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  for (int64_t i = 0; i < count; ++i) {
    const int64_t c = chunks(tensors[i].n);
    if (c == 0) continue;
    if (a.count == kMaxTensors || blocks + c > kMaxGrid) {
      HIP_TRY(run_step(a, blocks, o, master, st));
      a.count = 0;
      blocks = 0;
    }
    a.t[a.count] = tensors[i];
    a.first[a.count++] = (uint32_t)blocks;
    blocks += c;
  }
  if (a.count > 0) HIP_TRY(run_step(a, blocks, o, master, st));
  return DORA_OK;
}

DORA_API size_t dora_grad_norm_workspace_bytes(const dora_adamw_tensor* tensors, int64_t count) {
  if (check_tensors(tensors, count) != DORA_OK) return 0;
  int64_t parts = 0;
  for (int64_t i = 0; i < count; ++i) parts += chunks(tensors[i].n);
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
  int64_t done = 0, blocks = 0;
  NormArgs a;
  a.count = 0;
  auto flush = [&]() -> hipError_t {
    if (a.count == 0) return hipSuccess;
    LaunchTimer timer("grad_norm", st);
    if (grad_dtype == DORA_BF16)
      hipLaunchKernelGGL((dora_grad_norm_parts<true>), dim3((unsigned)blocks), dim3(kThreads), 0,
                         st, a, part + done);
    else
      hipLaunchKernelGGL((dora_grad_norm_parts<false>), dim3((unsigned)blocks), dim3(kThreads), 0,
                         st, a, part + done);
    done += blocks;
    blocks = 0;
    a.count = 0;
    return hipGetLastError();
  };
  for (int64_t i = 0; i < count; ++i) {
    const int64_t c = chunks(tensors[i].n);
    if (c == 0) continue;
    if (a.count == kMaxGrads || blocks + c > kMaxGrid) HIP_TRY(flush());
    a.g[a.count] = tensors[i].grad;
    a.n[a.count] = tensors[i].n;
    a.first[a.count++] = (uint32_t)blocks;
    blocks += c;
  }
  HIP_TRY(flush());
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
