// Layer norm over rows, forward and backward, with the reduction of the
// weight's and bias's gradients over the rows.
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

// One workgroup per row: mean, centred squares and output each take a pass.
template <bool BF>
__global__ __launch_bounds__(kThreads) void dora_layernorm_fwd_loop(
    const void* x_, int64_t ld, const void* w_, const void* b_, void* y_, float* mean_out,
    float* rstd_out, int64_t rows, int64_t D, float eps) {
  using E = Elem<BF>;
  using T = typename E::T;
  __shared__ float lds[2][kWaves];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
  const T* x = reinterpret_cast<const T*>(x_) + row * ld;
  const T* w = reinterpret_cast<const T*>(w_);
  const T* b = reinterpret_cast<const T*>(b_);
  T* y = reinterpret_cast<T*>(y_) + row * D;
  float sum = 0.f;
  for (int64_t j = (int64_t)threadIdx.x * E::kN; j < D; j += kThreads * E::kN) {
    float v[E::kN];
    load_part<BF>(x, j, D, 0.f, v);
#pragma unroll
    for (int q = 0; q < E::kN; ++q) sum += v[q];
  }
  block_sum<kWaves, 1>(&sum, lds[0]);
  const float mean = sum / (float)D;
  float sq = 0.f;
  for (int64_t j = (int64_t)threadIdx.x * E::kN; j < D; j += kThreads * E::kN) {
    float v[E::kN];
    load_part<BF>(x, j, D, mean, v);
#pragma unroll
    for (int q = 0; q < E::kN; ++q) sq = fmaf(v[q] - mean, v[q] - mean, sq);
  }
  block_sum<kWaves, 1>(&sq, lds[1]);
  const float rstd = 1.f / sqrtf(sq / (float)D + eps);
  if (threadIdx.x == 0) {
    if (mean_out) mean_out[row] = mean;
    if (rstd_out) rstd_out[row] = rstd;
  }
  for (int64_t j = (int64_t)threadIdx.x * E::kN; j < D; j += kThreads * E::kN) {
    float v[E::kN], wv[E::kN], bv[E::kN];
    load_part<BF>(x, j, D, 0.f, v);
#pragma unroll
    for (int q = 0; q < E::kN; ++q) wv[q] = 1.f, bv[q] = 0.f;
    if (w) load_part<BF>(w, j, D, 0.f, wv);
    if (b) load_part<BF>(b, j, D, 0.f, bv);
#pragma unroll
    for (int q = 0; q < E::kN; ++q) v[q] = fmaf((v[q] - mean) * rstd, wv[q], bv[q]);
    store_part<BF>(y, j, D, v);
  }
  }
}

// grad_x of one row per workgroup: a pass for the two means, a pass to write.
template <bool BF>
__global__ __launch_bounds__(kThreads) void dora_layernorm_bwd_x_loop(
    const void* gy_, int64_t ldg, const void* x_, int64_t ldx, const void* w_, const float* mean_in,
    const float* rstd_in, void* gx_, int64_t rows, int64_t D) {
  using E = Elem<BF>;
  using T = typename E::T;
  __shared__ float lds[2 * kWaves];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
  const T* gy = reinterpret_cast<const T*>(gy_) + row * ldg;
  const T* x = reinterpret_cast<const T*>(x_) + row * ldx;
  const T* w = reinterpret_cast<const T*>(w_);
  T* gx = reinterpret_cast<T*>(gx_) + row * D;
  const float mean = mean_in[row], rstd = rstd_in[row];
  float s[2] = {0.f, 0.f};
  for (int64_t j = (int64_t)threadIdx.x * E::kN; j < D; j += kThreads * E::kN) {
    float g[E::kN], v[E::kN], wv[E::kN];
    load_part<BF>(gy, j, D, 0.f, g);
    load_part<BF>(x, j, D, mean, v);
#pragma unroll
    for (int q = 0; q < E::kN; ++q) wv[q] = 1.f;
    if (w) load_part<BF>(w, j, D, 0.f, wv);
#pragma unroll
    for (int q = 0; q < E::kN; ++q) {
      const float h = g[q] * wv[q];
      s[0] += h;
      s[1] = fmaf(h, (v[q] - mean) * rstd, s[1]);
    }
  }
  block_sum<kWaves, 2>(s, lds);
  const float c1 = s[0] / (float)D, c2 = s[1] / (float)D;
  for (int64_t j = (int64_t)threadIdx.x * E::kN; j < D; j += kThreads * E::kN) {
    float g[E::kN], v[E::kN], wv[E::kN];
    load_part<BF>(gy, j, D, 0.f, g);
    load_part<BF>(x, j, D, mean, v);
#pragma unroll
    for (int q = 0; q < E::kN; ++q) wv[q] = 1.f;
    if (w) load_part<BF>(w, j, D, 0.f, wv);
#pragma unroll
    for (int q = 0; q < E::kN; ++q)
      v[q] = rstd * (fmaf(g[q], wv[q], -c1) - (v[q] - mean) * rstd * c2);
    store_part<BF>(gx, j, D, v);
  }
  __syncthreads();   // lds is written again for the next row
  }
}

// Column sums of gy xhat and gy over a block of rows, one thread per column:
// part[block][0 or 1][column].
template <bool BF>
__global__ __launch_bounds__(kThreads) void dora_layernorm_bwd_w_loop(
    const void* gy_, int64_t ldg, const void* x_, int64_t ldx, const float* mean_in,
    const float* rstd_in, float* part, int64_t rows, int64_t D, int64_t rows_per_block) {
  using E = Elem<BF>;
  using T = typename E::T;
  const int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (j >= D) return;
  const int64_t r0 = (int64_t)blockIdx.y * rows_per_block;
  const int64_t r1 = min(rows, r0 + rows_per_block);
  float gw = 0.f, gb = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float g = E::get(reinterpret_cast<const T*>(gy_) + r * ldg + j);
    const float v = E::get(reinterpret_cast<const T*>(x_) + r * ldx + j);
    gw = fmaf(g, (v - mean_in[r]) * rstd_in[r], gw);
    gb += g;
  }
  float* dst = part + (int64_t)blockIdx.y * 2 * D;
  dst[j] = gw;
  dst[D + j] = gb;
}

// grad_weight and grad_bias: the blocks' partial sums, added in order.
template <bool BF>
__global__ __launch_bounds__(kThreads) void dora_layernorm_bwd_w_finish(const float* part,
                                                                        int64_t blocks, void* gw,
                                                                        void* gb, int64_t D) {
  using E = Elem<BF>;
  using T = typename E::T;
  const int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (j >= D) return;
  if (gw) E::put(reinterpret_cast<T*>(gw) + j, sum_partials(part + j, blocks, 2 * D));
  if (gb) E::put(reinterpret_cast<T*>(gb) + j, sum_partials(part + D + j, blocks, 2 * D));
}

constexpr int64_t kMaxWidth = int64_t(1) << 22;
constexpr int64_t kMaxLd = int64_t(1) << 31;

bool shape_ok(const dora_layernorm_shape& s) {
  return s.rows >= 0 && s.rows < kMaxLd && s.width >= 1 && s.width < kMaxWidth &&
         s.ld_x >= s.width && s.ld_x < kMaxLd;
}
bool dtype_ok(const dora_layernorm_shape& s) { return s.dtype == DORA_F32 || s.dtype == DORA_BF16; }

int check_shape(const dora_layernorm_shape* s) {
  if (!s) return DORA_ERR_NULL;
  if (s->reserved != 0 || s->flags != 0 || !std::isfinite(s->eps) || s->eps < 0.f)
    return DORA_ERR_FLAGS;
  if (!dtype_ok(*s)) return DORA_ERR_DTYPE;
  if (!shape_ok(*s)) return DORA_ERR_SHAPE;
  return DORA_OK;
}

// Row blocks of the weight gradient's partial sums.
int64_t w_blocks(const dora_layernorm_shape& s) {
  return s.rows < 1 ? 0 : (s.rows + 31) / 32 < 256 ? (s.rows + 31) / 32 : 256;
}
size_t w_part_bytes(const dora_layernorm_shape& s) {
  return (size_t)w_blocks(s) * 2 * (size_t)s.width * 4;
}

template <bool BF>
hipError_t forward(const dora_layernorm_shape& s, const void* x, const void* w, const void* b,
                   void* y, float* mean, float* rstd, hipStream_t st) {
  LaunchTimer t("layernorm_fwd", st);
  hipLaunchKernelGGL((dora_layernorm_fwd_loop<BF>), dim3((unsigned)std::min(s.rows, kMaxGrid)),
                     dim3(kThreads), 0, st, x, s.ld_x, w, b, y, mean, rstd, s.rows, s.width, s.eps);
  return hipGetLastError();
}

template <bool BF>
hipError_t backward(const dora_layernorm_shape& s, const void* gy, const void* x, const void* w,
                    const float* mean, const float* rstd, void* gx, void* gw, void* gb, float* part,
                    hipStream_t st) {
  if (gx && s.rows > 0) {
    LaunchTimer t("layernorm_bwd_x", st);
    hipLaunchKernelGGL((dora_layernorm_bwd_x_loop<BF>), dim3((unsigned)std::min(s.rows, kMaxGrid)),
                       dim3(kThreads), 0, st, gy, s.ld_gy, x, s.ld_x, w, mean, rstd, gx, s.rows, s.width);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (!gw && !gb) return hipSuccess;
  const int64_t blocks = w_blocks(s);
  const unsigned cols = (unsigned)((s.width + kThreads - 1) / kThreads);
  if (blocks > 0) {
    LaunchTimer t("layernorm_bwd_w", st);
    hipLaunchKernelGGL((dora_layernorm_bwd_w_loop<BF>), dim3(cols, (unsigned)blocks),
                       dim3(kThreads), 0, st, gy, s.ld_gy, x, s.ld_x, mean, rstd, part, s.rows,
                       s.width, (s.rows + blocks - 1) / blocks);
    if (hipError_t e = hipGetLastError()) return e;
  }
  LaunchTimer t("layernorm_bwd_w_finish", st);
  hipLaunchKernelGGL((dora_layernorm_bwd_w_finish<BF>), dim3(cols), dim3(kThreads), 0, st, part,
                     blocks, gw, gb, s.width);
  return hipGetLastError();
}

}  // namespace
}  // namespace dora

using namespace dora;

extern "C" {

DORA_API size_t dora_layernorm_workspace_bytes(const dora_layernorm_shape* shape) {
  if (!shape || !dtype_ok(*shape) || !shape_ok(*shape)) return 0;
  return w_part_bytes(*shape);
}

DORA_API int dora_layernorm_forward(const dora_layernorm_shape* shape, const void* x,
                                    const void* weight, const void* bias, void* y, float* mean,
                                    float* rstd, void* hip_stream) {
  DORA_CHECK(check_shape(shape));
  const dora_layernorm_shape& s = *shape;
  const size_t e = s.dtype == DORA_BF16 ? 2 : 4;
  DORA_CHECK(check_elem(x, e, s.rows == 0));
  DORA_CHECK(check_elem(y, e, s.rows == 0));
  DORA_CHECK(check_elem(weight, e, true));
  DORA_CHECK(check_elem(bias, e, true));
  DORA_CHECK(check_elem(mean, 4, true));
  DORA_CHECK(check_elem(rstd, 4, true));
  if (s.rows == 0) return DORA_OK;
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  HIP_TRY(s.dtype == DORA_BF16 ? forward<true>(s, x, weight, bias, y, mean, rstd, st)
                               : forward<false>(s, x, weight, bias, y, mean, rstd, st));
  return DORA_OK;
}

DORA_API int dora_layernorm_backward(const dora_layernorm_shape* shape, const void* grad_y,
                                     const void* x, const void* weight, const float* mean,
                                     const float* rstd, void* grad_x, void* grad_weight,
                                     void* grad_bias, void* ws, size_t ws_bytes, void* hip_stream) {
  DORA_CHECK(check_shape(shape));
  const dora_layernorm_shape& s = *shape;
  if (s.ld_gy < s.width || s.ld_gy >= kMaxLd) return DORA_ERR_SHAPE;
  const size_t e = s.dtype == DORA_BF16 ? 2 : 4;
  const bool empty = s.rows == 0;
  DORA_CHECK(check_elem(grad_y, e, empty));
  DORA_CHECK(check_elem(x, e, empty));
  DORA_CHECK(check_elem(weight, e, true));
  DORA_CHECK(check_elem(mean, 4, empty));
  DORA_CHECK(check_elem(rstd, 4, empty));
  DORA_CHECK(check_elem(grad_x, e, true));
  DORA_CHECK(check_elem(grad_weight, e, true));
  DORA_CHECK(check_elem(grad_bias, e, true));
  if (grad_weight || grad_bias) DORA_CHECK(check_ws(ws, ws_bytes, w_part_bytes(s)));
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  float* part = reinterpret_cast<float*>(ws);
  HIP_TRY(s.dtype == DORA_BF16
              ? backward<true>(s, grad_y, x, weight, mean, rstd, grad_x, grad_weight, grad_bias,
                               part, st)
              : backward<false>(s, grad_y, x, weight, mean, rstd, grad_x, grad_weight, grad_bias,
                                part, st));
  return DORA_OK;
}

}  // extern "C"
