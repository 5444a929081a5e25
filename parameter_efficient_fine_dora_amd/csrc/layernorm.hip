// Layer norm over rows, forward and backward, with the reduction of the
// weight's and bias's gradients over the rows.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/dora.h"
#include "elem.h"
#include "entry.h"
#include "kernels.h"

namespace dora {
namespace {

// HIP holds the threads of a launch below 2^32: more rows than this share
// workgroups.
constexpr int64_t kMaxGrid = int64_t(1) << 21;

// ---- rows that fit a workgroup's registers --------------------------------------
// A workgroup of 64 to 1024 threads holds a row, kElems elements (or, past 16384
// elements, twice that) of it per thread in 16-byte vectors that the threads take
// in turn.  Memory is read once; mean and centred squares are sums over registers.
// What a width leaves past its last whole vector, at most 7 elements, is one
// more scalar of the first threads.  Vectors stay as they were loaded and are
// decoded where they are used: registers, not arithmetic, limit how many rows a
// CU has in flight.
constexpr int kElems = 16;

// This thread's share of a row of D elements.
template <bool BF, int THREADS, int NV>
struct Share {
  using E = Elem<BF>;
  using T = typename E::T;
  typename E::Vec v[NV];
  float t;
  // 32-bit offsets from a row's address, which all threads share
  __device__ static uint32_t at(int u) { return ((uint32_t)u * THREADS + threadIdx.x) * E::kN; }
  __device__ static uint32_t body(uint32_t D) { return D & ~(uint32_t)(E::kN - 1); }
  __device__ static bool has(int u, uint32_t D) { return at(u) < body(D); }
  __device__ static bool has_tail(uint32_t D) { return threadIdx.x < D - body(D); }
  __device__ void load(const T* row, uint32_t D) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      v[u] = typename E::Vec{0, 0, 0, 0};
      if (has(u, D)) v[u] = E::raw(row + at(u));
    }
    t = has_tail(D) ? E::get(row + body(D) + threadIdx.x) : 0.f;
  }
  // The second use of a share decodes it anew instead of keeping its decoded
  // elements across a barrier.
  __device__ void forget() {
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        auto r = v[u][d];
        asm volatile("" : "+v"(r));
        v[u][d] = r;
      }
  }
  __device__ void fill(float one) {   // every element that value (1 or 0)
    float f[E::kN];
#pragma unroll
    for (int q = 0; q < E::kN; ++q) f[q] = one;
#pragma unroll
    for (int u = 0; u < NV; ++u) v[u] = E::encode(f);
    t = one;
  }
};

template <bool BF, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void dora_layernorm_fwd(
    const void* x_, int64_t ld, const void* w_, const void* b_, void* y_, float* mean_out,
    float* rstd_out, int64_t rows, uint32_t D, float eps) {
  using E = Elem<BF>;
  using T = typename E::T;
  using S = Share<BF, THREADS, NV>;
  constexpr int kWaves = THREADS / 64;
  __shared__ float lds[2][kWaves];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    T* y = reinterpret_cast<T*>(y_) + row * D;
    S x, w, b;
    x.load(reinterpret_cast<const T*>(x_) + row * ld, D);
    if (w_)   // weight and bias are in flight during the reductions
      w.load(reinterpret_cast<const T*>(w_), D);
    else
      w.fill(1.f);
    if (b_)
      b.load(reinterpret_cast<const T*>(b_), D);
    else
      b.fill(0.f);
    float sum = x.t;   // absent elements are 0
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float v[E::kN];
      E::decode(x.v[u], v);
#pragma unroll
      for (int q = 0; q < E::kN; ++q) sum += v[q];
    }
    block_sum<kWaves, 1>(&sum, lds[0]);
    const float mean = sum / (float)D;
    x.forget();
    float sq = S::has_tail(D) ? (x.t - mean) * (x.t - mean) : 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float v[E::kN];
      E::decode(x.v[u], v);
      if (S::has(u, D)) {
#pragma unroll
        for (int q = 0; q < E::kN; ++q) sq = fmaf(v[q] - mean, v[q] - mean, sq);
      }
    }
    block_sum<kWaves, 1>(&sq, lds[1]);
    const float rstd = 1.f / sqrtf(sq / (float)D + eps);
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
    x.forget();
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float v[E::kN], wv[E::kN], bv[E::kN];
      E::decode(x.v[u], v);
      E::decode(w.v[u], wv);
      E::decode(b.v[u], bv);
#pragma unroll
      for (int q = 0; q < E::kN; ++q) v[q] = fmaf((v[q] - mean) * rstd, wv[q], bv[q]);
      if (S::has(u, D)) E::store(y + S::at(u), v);
    }
    if (S::has_tail(D))
      E::put(y + S::body(D) + threadIdx.x, fmaf((x.t - mean) * rstd, w.t, b.t));
  }
}

// grad_x, and with W the workgroup's share of grad_weight and grad_bias: its
// rows are blockIdx.x, blockIdx.x + gridDim.x, ...; every thread keeps the sums
// of its own columns in registers and writes them at the end as
// part[blockIdx.x][0 or 1][column].  The next row is loaded before this row's
// reduction, where registers allow (1024 threads have 128 each).
template <bool BF, int THREADS, int NV, bool W>
__global__ __launch_bounds__(THREADS) void dora_layernorm_bwd(
    const void* gy_, int64_t ldg, const void* x_, int64_t ldx, const void* w_, const float* mean_in,
    const float* rstd_in, void* gx_, float* part, int64_t rows, uint32_t D) {
  using E = Elem<BF>;
  using T = typename E::T;
  using S = Share<BF, THREADS, NV>;
  constexpr int kWaves = THREADS / 64;
  constexpr bool kAhead = THREADS < 1024 || 5 * 4 * NV + (W ? 2 * NV * E::kN : 0) <= 96;
  __shared__ float lds[2][2 * kWaves];
  S w, g, x, g_next, x_next;
  float mean_next = 0.f, rstd_next = 0.f;
  float gw[NV * E::kN], gb[NV * E::kN], gw_t = 0.f, gb_t = 0.f;
#pragma unroll
  for (int i = 0; i < NV * E::kN; ++i) gw[i] = gb[i] = 0.f;
  auto fetch = [&](int64_t row) {
    g_next.load(reinterpret_cast<const T*>(gy_) + row * ldg, D);
    x_next.load(reinterpret_cast<const T*>(x_) + row * ldx, D);
    mean_next = mean_in[row];
    rstd_next = rstd_in[row];
  };
  if (kAhead && blockIdx.x < rows) fetch(blockIdx.x);
  if (w_)
    w.load(reinterpret_cast<const T*>(w_), D);
  else
    w.fill(1.f);
  int buf = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, buf ^= 1) {
    w.forget();
    if (!kAhead) fetch(row);
    const float mean = mean_next, rstd = rstd_next;
    g = g_next;
    x = x_next;
    if (kAhead && row + gridDim.x < rows) fetch(row + gridDim.x);
    float s[2];   // absent elements have gy = 0
    {
      const float n = (x.t - mean) * rstd, h = g.t * w.t;
      gw_t = fmaf(g.t, n, gw_t);
      gb_t += g.t;
      s[0] = h;
      s[1] = h * n;
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float gv[E::kN], xv[E::kN], wv[E::kN];
      E::decode(g.v[u], gv);
      E::decode(x.v[u], xv);
      E::decode(w.v[u], wv);
#pragma unroll
      for (int q = 0; q < E::kN; ++q) {
        const float n = (xv[q] - mean) * rstd, h = gv[q] * wv[q];
        if (W) {
          gw[u * E::kN + q] = fmaf(gv[q], n, gw[u * E::kN + q]);
          gb[u * E::kN + q] += gv[q];
        }
        s[0] += h;
        s[1] = fmaf(h, n, s[1]);
      }
    }
    if (!gx_) continue;
    block_sum<kWaves, 2>(s, lds[buf]);
    const float c1 = s[0] / (float)D, c2 = s[1] / (float)D;
    T* gx = reinterpret_cast<T*>(gx_) + row * D;
    w.forget();
    g.forget();
    x.forget();
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float gv[E::kN], xv[E::kN], wv[E::kN];
      E::decode(g.v[u], gv);
      E::decode(x.v[u], xv);
      E::decode(w.v[u], wv);
#pragma unroll
      for (int q = 0; q < E::kN; ++q)
        gv[q] = rstd * (gv[q] * wv[q] - fmaf((xv[q] - mean) * rstd, c2, c1));
      if (S::has(u, D)) E::store(gx + S::at(u), gv);
    }
    if (S::has_tail(D))
      E::put(gx + S::body(D) + threadIdx.x,
             rstd * (g.t * w.t - fmaf((x.t - mean) * rstd, c2, c1)));
  }
  if (W) {
    float* dst = part + (int64_t)blockIdx.x * 2 * (int64_t)D;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (!S::has(u, D)) continue;
#pragma unroll
      for (int q = 0; q < E::kN; q += 4) {
        Elem<false>::store(dst + S::at(u) + q, gw + u * E::kN + q);
        Elem<false>::store(dst + D + S::at(u) + q, gb + u * E::kN + q);
      }
    }
    if (S::has_tail(D)) {
      dst[S::body(D) + threadIdx.x] = gw_t;
      dst[D + S::body(D) + threadIdx.x] = gb_t;
    }
  }
}

// ---- rows of any width: every step takes its own pass over memory ------------------
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

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

// grad_weight and grad_bias: the workgroups' partial sums added in order, 64
// columns of [grad_weight | grad_bias] per workgroup, 16 threads to a column.
template <bool BF>
__global__ __launch_bounds__(1024) void dora_layernorm_bwd_finish(const float* part, int64_t blocks,
                                                                  void* gw, void* gb, int64_t first,
                                                                  int64_t last, int64_t D) {
  using E = Elem<BF>;
  using T = typename E::T;
  __shared__ float lds[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = first + (int64_t)blockIdx.x * 64 + lane;
  const int64_t count = blocks > wave ? (blocks - wave + 15) / 16 : 0;
  if (c < last) lds[wave][lane] = sum_partials(part + (int64_t)wave * 2 * D + c, count, 16 * 2 * D);
  __syncthreads();
  if (wave != 0 || c >= last) return;
  float v = lds[0][lane];
#pragma unroll
  for (int i = 1; i < 16; ++i) v += lds[i][lane];
  if (c < D)
    E::put(reinterpret_cast<T*>(gw) + c, v);
  else
    E::put(reinterpret_cast<T*>(gb) + c - D, v);
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

// Threads that hold a row: kElems elements each, twice that past 16384
// elements; 0 for rows past 32768, which take the loops over memory.
int row_threads(int64_t D) {
  for (int t = 64; t <= 1024; t *= 2)
    if (D <= (int64_t)t * kElems) return t;
  return D <= 1024 * 2 * kElems ? 1024 : 0;
}
// Whether the backward's row kernel also sums the weight's gradient: past 16384
// elements its sums no longer fit beside the row, and gy and x are read again.
bool fused_sums(int64_t D) { return D <= 1024 * kElems; }

// Workgroups of the backward, which is also how many partial sums the weight's
// gradient has.  As many rounds of rows as it takes kCuThreads threads per CU,
// then the fewest workgroups with that many rounds.
constexpr int64_t kCus = 256;
constexpr int64_t kCuThreads = 1024;
int64_t bwd_blocks(const dora_layernorm_shape& s) {
  if (s.rows < 1) return 0;
  const int64_t most =
      fused_sums(s.width) ? kCus * std::max<int64_t>(1, kCuThreads / row_threads(s.width)) : kCus;
  const int64_t rounds = (s.rows + most - 1) / most;
  return (s.rows + rounds - 1) / rounds;
}
size_t w_part_bytes(const dora_layernorm_shape& s) {
  return (size_t)bwd_blocks(s) * 2 * (size_t)s.width * 4;
}

// f(threads, vectors) with the kernel's template arguments for rows of at most
// 16384 elements.
template <bool BF, typename F>
hipError_t with_threads(int64_t D, F f) {
  using std::integral_constant;
  integral_constant<int, kElems / Elem<BF>::kN> nv;
  switch (row_threads(D)) {
    case 64: return f(integral_constant<int, 64>(), nv);
    case 128: return f(integral_constant<int, 128>(), nv);
    case 256: return f(integral_constant<int, 256>(), nv);
    case 512: return f(integral_constant<int, 512>(), nv);
    default: return f(integral_constant<int, 1024>(), nv);
  }
}

template <bool BF>
hipError_t forward(const dora_layernorm_shape& s, const void* x, const void* w, const void* b,
                   void* y, float* mean, float* rstd, hipStream_t st) {
  constexpr int kWide = 2 * kElems / Elem<BF>::kN;
  const dim3 grid((unsigned)std::min(s.rows, kMaxGrid));
  LaunchTimer t("layernorm_fwd", st);
  if (row_threads(s.width) == 0) {
    hipLaunchKernelGGL((dora_layernorm_fwd_loop<BF>), grid, dim3(kThreads), 0, st, x, s.ld_x, w, b,
                       y, mean, rstd, s.rows, s.width, s.eps);
  } else if (s.width > 1024 * kElems) {
    hipLaunchKernelGGL((dora_layernorm_fwd<BF, 1024, kWide>), grid, dim3(1024), 0, st, x, s.ld_x, w,
                       b, y, mean, rstd, s.rows, (uint32_t)s.width, s.eps);
  } else {
    return with_threads<BF>(s.width, [&](auto threads, auto nv) {
      hipLaunchKernelGGL((dora_layernorm_fwd<BF, threads(), nv()>), grid, dim3(threads()), 0, st, x,
                         s.ld_x, w, b, y, mean, rstd, s.rows, (uint32_t)s.width, s.eps);
      return hipGetLastError();
    });
  }
  return hipGetLastError();
}

// grad_x alone, for rows past the fused kernel's.
template <bool BF>
hipError_t backward_x(const dora_layernorm_shape& s, const void* gy, const void* x, const void* w,
                      const float* mean, const float* rstd, void* gx, hipStream_t st) {
  constexpr int kWide = 2 * kElems / Elem<BF>::kN;
  const dim3 grid((unsigned)std::min(s.rows, kMaxGrid));
  LaunchTimer t("layernorm_bwd_x", st);
  if (row_threads(s.width) > 0)
    hipLaunchKernelGGL((dora_layernorm_bwd<BF, 1024, kWide, false>), grid, dim3(1024), 0, st, gy,
                       s.ld_gy, x, s.ld_x, w, mean, rstd, gx, nullptr, s.rows,
                       (uint32_t)s.width);
  else
    hipLaunchKernelGGL((dora_layernorm_bwd_x_loop<BF>), grid, dim3(kThreads), 0, st, gy, s.ld_gy, x,
                       s.ld_x, w, mean, rstd, gx, s.rows, s.width);
  return hipGetLastError();
}

template <bool BF>
hipError_t backward(const dora_layernorm_shape& s, const void* gy, const void* x, const void* w,
                    const float* mean, const float* rstd, void* gx, void* gw, void* gb, float* part,
                    hipStream_t st) {
  const bool sums = gw || gb;
  const int64_t blocks = bwd_blocks(s);
  if (s.rows > 0 && fused_sums(s.width)) {
    LaunchTimer t("layernorm_bwd", st);
    const hipError_t e = with_threads<BF>(s.width, [&](auto threads, auto nv) {
      if (sums)
        hipLaunchKernelGGL((dora_layernorm_bwd<BF, threads(), nv(), true>), dim3((unsigned)blocks),
                           dim3(threads()), 0, st, gy, s.ld_gy, x, s.ld_x, w, mean, rstd, gx, part,
                           s.rows, (uint32_t)s.width);
      else if (gx)
        hipLaunchKernelGGL((dora_layernorm_bwd<BF, threads(), nv(), false>),
                           dim3((unsigned)blocks), dim3(threads()), 0, st, gy, s.ld_gy, x, s.ld_x,
                           w, mean, rstd, gx, part, s.rows, (uint32_t)s.width);
      return hipGetLastError();
    });
    if (e) return e;
  } else if (s.rows > 0) {
    if (gx)
      if (hipError_t e = backward_x<BF>(s, gy, x, w, mean, rstd, gx, st)) return e;
    if (sums) {
      LaunchTimer t("layernorm_bwd_w", st);
      const unsigned cols = (unsigned)((s.width + kThreads - 1) / kThreads);
      hipLaunchKernelGGL((dora_layernorm_bwd_w_loop<BF>), dim3(cols, (unsigned)blocks),
                         dim3(kThreads), 0, st, gy, s.ld_gy, x, s.ld_x, mean, rstd, part, s.rows,
                         s.width, (s.rows + blocks - 1) / blocks);
      if (hipError_t e = hipGetLastError()) return e;
    }
  }
  if (!sums) return hipSuccess;
  LaunchTimer t("layernorm_bwd_finish", st);
  const int64_t first = gw ? 0 : s.width, last = gb ? 2 * s.width : s.width;
  hipLaunchKernelGGL((dora_layernorm_bwd_finish<BF>), dim3((unsigned)((last - first + 63) / 64)),
                     dim3(1024), 0, st, part, blocks, gw, gb, first, last, s.width);
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
