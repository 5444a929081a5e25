// Layer norm over rows, forward and backward, with the reduction of the
// weight's and bias's gradients over the rows.
//   y      = xhat weight + bias, xhat = (x - mean) rstd,
//            rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   grad_x = rstd (h - mean(h) - xhat mean(h xhat)), h = grad_y weight
//   grad_weight = sum over rows of grad_y xhat, grad_bias = sum of grad_y
// All sums are float32 in an order that depends on sizes alone; results are
// rounded once, to the tensors' type.  Memory bounds both directions where rows
// are many: the forward reads and writes each element once (2048 x 6144 bf16: 10.7
// us a pass, 4.7 TB/s), the backward reads two and writes one (4096 x 8192 bf16: 35
// us, 6.2 TB/s with its partial sums, and 5 us to add those; 1031 x 5121 float32:
// 15 and 4 us; grad_x alone, with neither: 34 and 12 us a pass).  One row of 8192 is
// a launch's latency, 3 us.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/dora_finetune.h"
#include "checks.h"
#include "elem.h"
#include "kernels.h"

namespace dora {
namespace {

// HIP holds the threads of a launch below 2^32: more rows than this share
// workgroups.
constexpr int64_t kMaxGrid = int64_t(1) << 21;

// ---- rows that fit a workgroup's registers --------------------------------------
// A row is held by as many waves as take kElems elements (wide rows: twice that) of
// it per thread, in 16-byte vectors that the threads take in turn.
// Memory is read once; mean and centred squares are sums over registers.  What a
// width leaves past its last whole vector, at most 7 elements, is one more scalar
// of the first threads.  Vectors stay as they were loaded and are
// decoded where they are used: registers, not arithmetic, limit how many rows a
// CU has in flight.
constexpr int kElems = 16;

// This thread's share of a row of D elements.
template <bool BF, int THREADS, int NV>
struct Share {
  using E = Elem<BF>;
  using T = typename E::T;
  typename E::Vec v[NV];
  T tail;   // undecoded too: a use right after its load would wait for every load
  // 32-bit offsets from a row's address, which all threads share
  __device__ static uint32_t lane() { return threadIdx.x % THREADS; }
  __device__ static uint32_t at(int u) { return ((uint32_t)u * THREADS + lane()) * E::kN; }
  __device__ static uint32_t body(uint32_t D) { return D & ~(uint32_t)(E::kN - 1); }
  __device__ static bool has(int u, uint32_t D) { return at(u) < body(D); }
  __device__ static bool has_tail(uint32_t D) { return lane() < D - body(D); }
  __device__ void load(const T* row, uint32_t D) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      v[u] = typename E::Vec{0, 0, 0, 0};
      if (has(u, D)) v[u] = E::raw(row + at(u));
    }
    tail = 0;
    if (has_tail(D)) tail = row[body(D) + lane()];
  }
  // Vector u decoded, not before `after` is known: the second use of a share does
  // not keep its decoded elements from the first, and one vector's elements are
  // decoded at a time.
  __device__ void decode(int u, float* out, float& after) {
    typename E::Vec r = v[u];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      auto e = r[d];
      asm volatile("" : "+v"(e), "+v"(after));
      r[d] = e;
    }
    E::decode(r, out);
  }
  __device__ float t() const { return E::get(&tail); }
  __device__ void fill(float one) {   // every element that value (1 or 0)
    float f[E::kN];
#pragma unroll
    for (int q = 0; q < E::kN; ++q) f[q] = one;
#pragma unroll
    for (int u = 0; u < NV; ++u) v[u] = E::encode(f);
    E::put(&tail, one);
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
    float sum = x.t();   // absent elements are 0
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float v[E::kN];
      x.decode(u, v, sum);
#pragma unroll
      for (int q = 0; q < E::kN; ++q) sum += v[q];
    }
    block_sum<kWaves, 1>(&sum, lds[0]);
    float mean = sum / (float)D;
    float sq = S::has_tail(D) ? (x.t() - mean) * (x.t() - mean) : 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float v[E::kN];
      x.decode(u, v, sq);
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
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float v[E::kN], wv[E::kN], bv[E::kN];
      x.decode(u, v, mean);
      w.decode(u, wv, mean);
      b.decode(u, bv, mean);
#pragma unroll
      for (int q = 0; q < E::kN; ++q) v[q] = fmaf((v[q] - mean) * rstd, wv[q], bv[q]);
      if (S::has(u, D)) E::store(y + S::at(u), v);
    }
    if (S::has_tail(D))
      E::put(y + S::body(D) + S::lane(), fmaf((x.t() - mean) * rstd, w.t(), b.t()));
  }
}

// grad_x, and with W the workgroup's share of grad_weight and grad_bias.  A
// workgroup is a CU's: as many waves as its registers hold (bf16 12, float32 8),
// R rows at a time, THREADS threads to a row.  bf16 rows past 8192 elements are one
// row of 5 to 8 waves that hold twice as much (2048 x 16384: 49 us against 81 in two
// passes); float32 ones would spill.  Every thread keeps the sums of its
// own columns in registers over all its rows, and at the end the R rows' threads
// add theirs through LDS: part[blockIdx.x][0 or 1][column], as few partial sums as
// there are CUs.  The next rows are loaded before this row's reduction.  A row
// costs a CU about 20 operations an element, half of what memory takes, and
// waits twice for its reductions: several rows at a time fill those gaps.
constexpr int kMaxBwdThreads = 512;   // of a row
constexpr int bwd_rows(bool bf, int threads, bool wide) {
  // rows of one or two waves leave sums of 12 rows to add for little: 8 waves
  return wide ? 1 : (bf && threads > 128 ? 12 : 8) * 64 / threads;
}
// Rows fetched ahead: two where one row's waves leave registers for it (4096 x 8192
// bf16: 53.5 us against 54.7 with one where the GPU is waited for after every pass,
// 43.9 against 43.3 among others; three take longer, and float32 loses with two,
// 1031 x 5121 21 us against 20).
constexpr int bwd_ahead(bool bf, int threads, bool wide) {
  return bf && !wide && threads > 384 ? 2 : 1;
}
template <bool BF, int THREADS, int NV, bool W, bool GX>
__global__ __launch_bounds__(bwd_rows(BF, THREADS, NV * Elem<BF>::kN > kElems) * THREADS) void dora_layernorm_bwd(
    const void* gy_, int64_t ldg, const void* x_, int64_t ldx, const void* w_, const float* mean_in,
    const float* rstd_in, void* gx_, float* part, int64_t rows, uint32_t D) {
  using E = Elem<BF>;
  using T = typename E::T;
  using S = Share<BF, THREADS, NV>;
  constexpr bool kWide = NV * E::kN > kElems;
  constexpr int R = bwd_rows(BF, THREADS, kWide);
  constexpr int kWaves = THREADS / 64;
  __shared__ float lds[2][R][2 * kWaves];
  __shared__ __align__(16) float comb[W && R > 1 ? R : 1][W && R > 1 ? THREADS * NV * E::kN : 4];
  const int sub = __builtin_amdgcn_readfirstlane((int)threadIdx.x / THREADS);   // per wave
  constexpr int kAhead = bwd_ahead(BF, THREADS, kWide);
  // vectors that every thread has, from the narrowest row of so many threads
  constexpr int kFull = (THREADS - 64) * NV / THREADS;
  S w, g, x, g_next[kAhead], x_next[kAhead];
  float mean_next[kAhead], rstd_next[kAhead];
  float gw[NV * E::kN], gb[NV * E::kN], gw_t = 0.f, gb_t = 0.f;
#pragma unroll
  for (int i = 0; i < NV * E::kN; ++i) gw[i] = gb[i] = 0.f;
  const int64_t stride = (int64_t)gridDim.x * R;
  // rows past the last load as zeros, which add nothing
  auto fetch = [&](int64_t row, int slot) {
    const bool valid = row < rows;
    const int64_t at = valid ? row : 0;
    const uint32_t n = valid ? D : 0;
    g_next[slot].load(reinterpret_cast<const T*>(gy_) + at * ldg, n);
    x_next[slot].load(reinterpret_cast<const T*>(x_) + at * ldx, n);
    mean_next[slot] = valid ? mean_in[row] : 0.f;
    rstd_next[slot] = valid ? rstd_in[row] : 0.f;
  };
  int64_t row = (int64_t)blockIdx.x * R + sub;
#pragma unroll
  for (int slot = 0; slot < kAhead; ++slot) fetch(row + slot * stride, slot);
  if (w_)
    w.load(reinterpret_cast<const T*>(w_), D);
  else
    w.fill(1.f);
  int buf = 0;
  int64_t first = (int64_t)blockIdx.x * R;
  auto turn = [&](int slot, bool all) {   // all: every wave has a row
    const float mean = mean_next[slot], rstd = rstd_next[slot];
    g = g_next[slot];
    x = x_next[slot];
    if (first + kAhead * stride < rows) fetch(row + kAhead * stride, slot);
    // absent elements have x = gy = 0 and take 0 for their mean: (0 - mean) rstd may
    // be infinite
    float s[2];
    {
      const float n = (x.t() - (S::has_tail(D) ? mean : 0.f)) * rstd, h = g.t() * w.t();
      gw_t = fmaf(g.t(), n, gw_t);
      gb_t += g.t();
      s[0] = h;
      s[1] = h * n;
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float gv[E::kN], xv[E::kN], wv[E::kN];
      g.decode(u, gv, s[0]);
      x.decode(u, xv, s[0]);
      w.decode(u, wv, s[0]);
      const float mu = u < kFull || S::has(u, D) ? mean : 0.f;
#pragma unroll
      for (int q = 0; q < E::kN; ++q) {
        const float n = (xv[q] - mu) * rstd, h = gv[q] * wv[q];
        if (W) {
          gw[u * E::kN + q] = fmaf(gv[q], n, gw[u * E::kN + q]);
          gb[u * E::kN + q] += gv[q];
        }
        s[0] += h;
        s[1] = fmaf(h, n, s[1]);
      }
    }
    if (!GX) return;
    group_sum<kWaves, 2>(s, lds[buf][sub], threadIdx.x % THREADS);
    if (!all && row >= rows) return;
    const float c2 = s[1] / (float)D;
    float c1 = s[0] / (float)D;
    T* gx = reinterpret_cast<T*>(gx_) + row * D;
    if (S::has_tail(D))
      E::put(gx + S::body(D) + S::lane(),
             rstd * (g.t() * w.t() - fmaf((x.t() - mean) * rstd, c2, c1)));
    typename E::Vec zeroth;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float gv[E::kN], xv[E::kN], wv[E::kN];
      g.decode(u, gv, c1);
      x.decode(u, xv, c1);
      w.decode(u, wv, c1);
#pragma unroll
      for (int q = 0; q < E::kN; ++q)
        gv[q] = rstd * (gv[q] * wv[q] - fmaf((xv[q] - mean) * rstd, c2, c1));
      typename E::Vec out = E::encode(gv);
      if (u == 0) zeroth = out;
      if (kFull > 0) {
        // stores without a branch: a thread that lacks the vector repeats its first
        const bool in = u < kFull || S::has(u, D);
#pragma unroll
        for (int d = 0; d < 4; ++d) out[d] = in ? out[d] : zeroth[d];
        E::store_raw(gx + (in ? S::at(u) : S::at(0)), out);
      } else if (S::has(u, D)) {
        E::store_raw(gx + S::at(u), out);
      }
    }
  };
  // Every thread of the workgroup takes the same number of turns.  Where all have a
  // row no branch skips a vector's store: the wait for the next row's loads then
  // counts the stores behind them, instead of waiting for those too (4096 x 8192
  // bf16: 45 us against 50).
  static_assert(R == 1 || kAhead == 1, "a last turn without rows for all");
  bool more = first + R <= rows;
  while (more) {
#pragma unroll
    for (int slot = 0; slot < kAhead; ++slot) {
      turn(slot, true);
      first += stride;
      row += stride;
      buf ^= 1;
      more = first + R <= rows;
      if (!more) break;
    }
  }
  if (R > 1 && first < rows) turn(0, false);
  if (!W) return;
  float* dst = part + (int64_t)blockIdx.x * 2 * (int64_t)D;
  auto put = [&](float* to, const float* v, float t) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (!S::has(u, D)) continue;
#pragma unroll
      for (int q = 0; q < E::kN; q += 4) Elem<false>::store(to + S::at(u) + q, v + u * E::kN + q);
    }
    if (S::has_tail(D)) to[S::body(D) + S::lane()] = t;
  };
  if (R == 1) {
    put(dst, gw, gw_t);
    put(dst + D, gb, gb_t);
    return;
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    put(comb[sub], half ? gb : gw, half ? gb_t : gw_t);
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < D; c += R * THREADS) {
      float v = comb[0][c];
#pragma unroll
      for (int r = 1; r < (W ? R : 1); ++r) v += comb[r][c];
      dst[(int64_t)half * D + c] = v;
    }
    __syncthreads();
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

// Backward of still wider rows, where a row's sums and the weight gradient's do not fit
// one thread's registers: a workgroup per row forms the two means, and a second
// kernel goes down columns.  Memory is read twice and written once (1024 x 27648
// bf16: 66 us, 4.3 TB/s).
template <bool BF>
__global__ __launch_bounds__(kThreads) void dora_layernorm_bwd_means(
    const void* gy_, int64_t ldg, const void* x_, int64_t ldx, const void* w_, const float* mean_in,
    const float* rstd_in, float2* means, int64_t rows, int64_t D) {
  using E = Elem<BF>;
  using T = typename E::T;
  __shared__ float lds[2][2 * kWaves];
  constexpr int kU = 4, kStep = kThreads * E::kN;   // vectors in flight, and apart
  int buf = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, buf ^= 1) {
    const T* gy = reinterpret_cast<const T*>(gy_) + row * ldg;
    const T* x = reinterpret_cast<const T*>(x_) + row * ldx;
    const T* w = reinterpret_cast<const T*>(w_);
    const float mean = mean_in[row], rstd = rstd_in[row];
    float s[2] = {0.f, 0.f};
    auto add = [&](const float* g, const float* v, const float* wv) {
#pragma unroll
      for (int q = 0; q < E::kN; ++q) {
        const float h = g[q] * wv[q];
        s[0] += h;
        s[1] = fmaf(h, (v[q] - mean) * rstd, s[1]);
      }
    };
    float wv[E::kN];
#pragma unroll
    for (int q = 0; q < E::kN; ++q) wv[q] = 1.f;
    int64_t j = (int64_t)threadIdx.x * E::kN;
    for (int64_t end = kU * kStep; end <= D; end += kU * kStep, j += kU * kStep) {
      typename E::Vec g[kU], v[kU], wr[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (w) wr[u] = E::raw(w + j + u * kStep);
        g[u] = E::raw(gy + j + u * kStep);
        v[u] = E::raw(x + j + u * kStep);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        float gv[E::kN], xv[E::kN];
        E::decode(g[u], gv);
        E::decode(v[u], xv);
        if (w) E::decode(wr[u], wv);
        add(gv, xv, wv);
      }
    }
    for (; j < D; j += kStep) {
      float gv[E::kN], xv[E::kN];
      load_part<BF>(gy, j, D, 0.f, gv);
      load_part<BF>(x, j, D, mean, xv);
      if (w) load_part<BF>(w, j, D, 0.f, wv);
      add(gv, xv, wv);
    }
    block_sum<kWaves, 2>(s, lds[buf]);
    if (threadIdx.x == 0) means[row] = float2{s[0] / (float)D, s[1] / (float)D};
  }
}

// Columns [blockIdx.x * kThreads * kN, ...) of the rows [blockIdx.y *
// rows_per_block, ...): grad_x from the rows' means, and the block's sums of gy
// xhat and gy as part[blockIdx.y][0 or 1][column].
template <bool BF>
__global__ __launch_bounds__(kThreads) void dora_layernorm_bwd_columns(
    const void* gy_, int64_t ldg, const void* x_, int64_t ldx, const void* w_, const float* mean_in,
    const float* rstd_in, const float2* means, void* gx_, float* part, int64_t rows, int64_t D,
    int64_t rows_per_block) {
  using E = Elem<BF>;
  using T = typename E::T;
  constexpr int U = 4;   // rows in flight
  const int64_t j = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * E::kN;
  if (j >= D) return;
  const T* gy = reinterpret_cast<const T*>(gy_);
  const T* x = reinterpret_cast<const T*>(x_);
  T* gx = reinterpret_cast<T*>(gx_);
  const int64_t r0 = (int64_t)blockIdx.y * rows_per_block;
  const int64_t r1 = min(rows, r0 + rows_per_block);
  float w[E::kN], gw[E::kN], gb[E::kN];
#pragma unroll
  for (int q = 0; q < E::kN; ++q) w[q] = 1.f, gw[q] = gb[q] = 0.f;
  if (w_) load_part<BF>(reinterpret_cast<const T*>(w_), j, D, 0.f, w);
  auto row = [&](int64_t r, float* g, float* v) {
    const float mean = mean_in[r], rstd = rstd_in[r];
    const float2 c = gx ? means[r] : float2{0.f, 0.f};
#pragma unroll
    for (int q = 0; q < E::kN; ++q) {
      const float n = (v[q] - mean) * rstd;
      gw[q] = fmaf(g[q], n, gw[q]);
      gb[q] += g[q];
      g[q] = rstd * (g[q] * w[q] - fmaf(n, c.y, c.x));
    }
    if (gx) store_part<BF>(gx + r * D, j, D, g);
  };
  int64_t r = r0;
  if (j + E::kN <= D) {
    for (; r + U <= r1; r += U) {
      typename E::Vec g[U], v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        g[u] = E::raw(gy + (r + u) * ldg + j);
        v[u] = E::raw(x + (r + u) * ldx + j);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float gv[E::kN], xv[E::kN];
        E::decode(g[u], gv);
        E::decode(v[u], xv);
        row(r + u, gv, xv);
      }
    }
  }
  for (; r < r1; ++r) {
    float gv[E::kN], xv[E::kN];
    load_part<BF>(gy + r * ldg, j, D, 0.f, gv);
    load_part<BF>(x + r * ldx, j, D, 0.f, xv);
    row(r, gv, xv);
  }
  if (part) {
    float* dst = part + (int64_t)blockIdx.y * 2 * D;
#pragma unroll
    for (int q = 0; q < E::kN; q += 4) {
      store_part<false>(dst, j + q, D, gw + q);
      store_part<false>(dst + D, j + q, D, gb + q);
    }
  }
}

// grad_weight and grad_bias: the workgroups' partial sums added in order, 64
// columns of [grad_weight | grad_bias] per workgroup, 16 threads to a column
// (256 partial sums of 2 x 8192 columns, 16.8 MB from the last-level cache: 4.8 us).
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

// Threads that hold a row of the backward: whole waves, kElems elements a thread, or
// twice that for wide rows (bf16 only: float32 ones spill).
bool bwd_wide(int64_t D) { return D > kMaxBwdThreads * kElems; }
int row_threads(int64_t D) {
  const int64_t per = 64 * kElems * (bwd_wide(D) ? 2 : 1);
  return (int)((D + per - 1) / per) * 64;
}
// The forward's threads: powers of two, whose idle lanes are waves more in flight
// (2048 x 6144 bf16: 10.7 us a pass against 11.3).
int fwd_threads(int64_t D) {
  int t = 64;
  while ((int64_t)t * kElems < D) t *= 2;
  return t;
}
// Longer rows the forward holds in 1024 threads, up to twice kElems elements each
// (in float32 that many, with their weights, spill); beyond, it loops over memory.
int64_t fwd_most(bool bf) { return (bf ? 2 : 1) * 1024 * kElems; }
// Rows that the backward holds in registers beside the weight gradient's sums.
bool bwd_in_registers(const dora_layernorm_shape& s) {
  return s.width <= kMaxBwdThreads * kElems * (s.dtype == DORA_BF16 ? 2 : 1);
}
static_assert(DORA_LAYERNORM_NO_WS_WIDTH(DORA_F32) == kMaxBwdThreads * kElems &&
                  DORA_LAYERNORM_NO_WS_WIDTH(DORA_BF16) == 2 * kMaxBwdThreads * kElems,
              "rows held in registers need no workspace for grad_x alone");

// Row blocks of the backward, which is also how many partial sums the weight's
// gradient has.  In registers: one workgroup per CU, or as few as take no more
// rounds.  Down columns: workgroups enough for four per CU, none under 16 rows.
constexpr int64_t kCus = 256;
int64_t bwd_blocks(const dora_layernorm_shape& s) {
  if (s.rows < 1) return 0;
  const bool bf = s.dtype == DORA_BF16;
  if (bwd_in_registers(s)) {
    const int64_t at_once = bwd_rows(bf, row_threads(s.width), bwd_wide(s.width));
    const int64_t groups = (s.rows + at_once - 1) / at_once;
    const int64_t rounds = (groups + kCus - 1) / kCus;
    return (groups + rounds - 1) / rounds;
  }
  const int64_t per = kThreads * (bf ? 8 : 4);
  const int64_t cols = (s.width + per - 1) / per;
  const int64_t want = std::max<int64_t>(1, 4 * kCus / cols);
  const int64_t rows = std::max<int64_t>(16, (s.rows + want - 1) / want);
  return (s.rows + rows - 1) / rows;
}
size_t part_bytes(const dora_layernorm_shape& s) {
  return ((size_t)bwd_blocks(s) * 2 * (size_t)s.width * 4 + 15) / 16 * 16;
}
// The workspace: the weight gradient's partial sums, then the means of wide rows.
size_t ws_bytes_for(const dora_layernorm_shape& s) {
  return part_bytes(s) + (bwd_in_registers(s) ? 0 : (size_t)s.rows * sizeof(float2));
}

// f(threads) with a row kernel's template argument.
template <typename F>
hipError_t with_threads(int threads, F f) {
  using std::integral_constant;
  switch (threads) {
    case 64: return f(integral_constant<int, 64>());
    case 128: return f(integral_constant<int, 128>());
    case 256: return f(integral_constant<int, 256>());
    case 512: return f(integral_constant<int, 512>());
    default: return hipErrorInvalidValue;
  }
}
template <typename F>
hipError_t with_any_threads(int threads, F f) {
  using std::integral_constant;
  switch (threads) {
    case 192: return f(integral_constant<int, 192>());
    case 320: return f(integral_constant<int, 320>());
    case 384: return f(integral_constant<int, 384>());
    case 448: return f(integral_constant<int, 448>());
    default: return with_threads(threads, f);
  }
}

template <bool BF>
hipError_t forward(const dora_layernorm_shape& s, const void* x, const void* w, const void* b,
                   void* y, float* mean, float* rstd, hipStream_t st) {
  constexpr int NV = kElems / Elem<BF>::kN;
  const dim3 grid((unsigned)std::min(s.rows, kMaxGrid));
  LaunchTimer t("layernorm_fwd", st);
  const uint32_t D = (uint32_t)s.width;
  if (D > fwd_most(BF)) {
    hipLaunchKernelGGL((dora_layernorm_fwd_loop<BF>), grid, dim3(kThreads), 0, st, x, s.ld_x, w, b,
                       y, mean, rstd, s.rows, s.width, s.eps);
  } else if (D > 1024 * kElems) {
    if constexpr (BF)
      hipLaunchKernelGGL((dora_layernorm_fwd<BF, 1024, 2 * NV>), grid, dim3(1024), 0, st, x, s.ld_x,
                         w, b, y, mean, rstd, s.rows, D, s.eps);
  } else if (D > kMaxBwdThreads * kElems) {
    hipLaunchKernelGGL((dora_layernorm_fwd<BF, 1024, NV>), grid, dim3(1024), 0, st, x, s.ld_x, w, b,
                       y, mean, rstd, s.rows, D, s.eps);
  } else {
    return with_threads(fwd_threads(D), [&](auto threads) {
      hipLaunchKernelGGL((dora_layernorm_fwd<BF, threads(), NV>), grid, dim3(threads()), 0, st, x,
                         s.ld_x, w, b, y, mean, rstd, s.rows, D, s.eps);
      return hipGetLastError();
    });
  }
  return hipGetLastError();
}

template <bool BF>
hipError_t backward(const dora_layernorm_shape& s, const void* gy, const void* x, const void* w,
                    const float* mean, const float* rstd, void* gx, void* gw, void* gb, void* ws,
                    hipStream_t st) {
  constexpr int NV = kElems / Elem<BF>::kN;
  const bool sums = gw || gb;
  const int64_t blocks = bwd_blocks(s);
  float* part = sums ? reinterpret_cast<float*>(ws) : nullptr;
  if (s.rows > 0 && (gx || sums) && bwd_in_registers(s)) {
    LaunchTimer t("layernorm_bwd", st);
    auto launch = [&](auto kernel, int threads) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(threads), 0, st, gy, s.ld_gy, x,
                         s.ld_x, w, mean, rstd, gx, part, s.rows, (uint32_t)s.width);
      return hipGetLastError();
    };
    auto pick = [&](auto threads, auto vectors) {
      constexpr int T = threads(), V = vectors();
      constexpr int block = bwd_rows(BF, T, V > NV) * T;
      if (!gx) return launch(dora_layernorm_bwd<BF, T, V, true, false>, block);
      return sums ? launch(dora_layernorm_bwd<BF, T, V, true, true>, block)
                  : launch(dora_layernorm_bwd<BF, T, V, false, true>, block);
    };
    const hipError_t e = with_any_threads(row_threads(s.width), [&](auto threads) {
      using std::integral_constant;
      if constexpr (BF && threads() >= 320)
        if (bwd_wide(s.width)) return pick(threads, integral_constant<int, 2 * NV>());
      return pick(threads, integral_constant<int, NV>());
    });
    if (e) return e;
  } else if (s.rows > 0 && (gx || sums)) {
    float2* means = gx ? reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(ws) + part_bytes(s))
                       : nullptr;
    if (gx) {
      LaunchTimer t("layernorm_bwd_means", st);
      hipLaunchKernelGGL((dora_layernorm_bwd_means<BF>),
                         dim3((unsigned)std::min(s.rows, kMaxGrid)), dim3(kThreads), 0, st, gy,
                         s.ld_gy, x, s.ld_x, w, mean, rstd, means, s.rows, s.width);
      if (hipError_t e = hipGetLastError()) return e;
    }
    LaunchTimer t("layernorm_bwd_columns", st);
    const int64_t per = kThreads * Elem<BF>::kN;
    hipLaunchKernelGGL((dora_layernorm_bwd_columns<BF>),
                       dim3((unsigned)((s.width + per - 1) / per), (unsigned)blocks),
                       dim3(kThreads), 0, st, gy, s.ld_gy, x, s.ld_x, w, mean, rstd, means, gx,
                       part, s.rows, s.width, (s.rows + blocks - 1) / blocks);
    if (hipError_t e = hipGetLastError()) return e;
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
  return ws_bytes_for(*shape);
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
  // rows held in registers need none for grad_x alone
  if (grad_weight || grad_bias || (grad_x && !bwd_in_registers(s)))
    DORA_CHECK(check_ws(ws, ws_bytes, ws_bytes_for(s)));
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  HIP_TRY(s.dtype == DORA_BF16
              ? backward<true>(s, grad_y, x, weight, mean, rstd, grad_x, grad_weight, grad_bias,
                               ws, st)
              : backward<false>(s, grad_y, x, weight, mean, rstd, grad_x, grad_weight, grad_bias,
                                ws, st));
  return DORA_OK;
}

}  // extern "C"
