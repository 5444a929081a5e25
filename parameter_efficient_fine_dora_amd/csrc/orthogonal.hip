// Orthogonalised updates: X_0 = X / (|X|_F + eps), then for each step
//   X <- P X,  P = a + b S + c S^2,  S = X X^T   (n x n, n the shorter side of X, m the longer).
//
// Everything between the first S and the last product stays n x n.  The P of all steps are
// polynomials of the first S, so they commute, and
//   S <- P S P,  Q <- P Q,  X_last = Q X_0
// replace two products with X in every step (4 n^2 m flops each way round) by one half of one
// (S is symmetric) and one at the end; adapters have n of 16 to 400 against m of thousands.  The
// n x n products are symmetric too: only tiles on and above the diagonal are computed.
//
// Precision.  A step multiplies small singular values by a (3.4445 as usually chosen), so five
// steps raise an error in S of E (relative to |X|_F^2) to |b/a| sum_j prod_{i<j} a_i^2 E = 3e4 E in
// the directions below 2^-9 of the norm.  All n x n matrices are therefore held as two half
// precision numbers, hi + lo (22 bits or more: the hi product and both cross products go through
// the matrix cores, the lo lo product is below 2^-22), scaled by powers of two into half's range;
// sums are float32.  For bf16 results that is enough.  Others form the product Q X on the way, before
// the factor passes what they allow (kMostExact, kMostUpdate), and S anew from it.
// A bf16 X is one half precision number exactly (its bits below 2^-38 of its largest element are
// left out), a float32 X and every update are hi + lo, scaled by a power of two that X's largest element
// asks for, so that any finite X is held to 22 bits.  (That costs a pass over gradient and momentum.
// Two bf16 numbers, which hold float32's range, would save it for bf16 parameters, on one card 24 rank-384
// layers' step 1.42 ms instead of 1.62, but keep 16 bits, raised 485 times, and their squares overflow from
// 2^104 eps on.)
//
// Layout.  A "pair" row holds blocks of 32 columns: 32 hi, then 32 lo, so that the 128 bytes that
// a stage copies of a row are the hi and lo of 32 columns; a "single" row holds 64 columns there.
// X stays in its own order: where the sum runs down its rows (S of a tall matrix, Q X of a wide
// one) its numbers are turned as they are read from LDS.
//
// Many matrices share a launch: a step on the adapters of a model is 19 launches (bf16 parameters, five
// steps; up to 120 matrices of up to 12 sizes on one side of 64), and small matrices fill the chip together.
//
// n <= 64 (most adapters) takes another way: the n x n products of one matrix are one workgroup's, in
// LDS, S is summed by the pass that writes X, and Q X is not kept on the way but formed again where it
// is wanted.  Then a step is four launches (six with float32 masters), and memory bounds it.
#include <algorithm>
#include <cmath>
#include <type_traits>
#include <vector>

#include "../../include/dora_posttrain.h"
#include "checks.h"
#include "elem.h"
#include "kernels.h"
#include "launch_cut.h"

namespace dora {
namespace {

typedef _Float16 f16;
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t Rsrc;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kRowBytes = 128;       // of a row in one stage
constexpr int kPairBlock = 32;       // columns of a pair row's block
constexpr int kMaxGroups = 12;
constexpr int kMaxMatrices = 120;    // of one launch that needs their addresses
constexpr int kMaxSteps = 16;
constexpr int kMaxBlocks = 1024;     // workgroups that look for one matrix's largest element
// Parts of a sum over m: for n <= 64 one workgroup adds them, which costs 6 us for 64, and few
// workgroups cost more (16 x 200000: 337 us, with 32 parts 503).
constexpr int kMaxSplits = 64, kMaxParts = 32;

// ---- matrices of one size ---------------------------------------------------------------
// Offsets are bytes from a matrix's own part of the workspace.
struct Group {
  int n, m;            // shorter and longer side
  int ne;              // n in whole blocks of 64: what sums over n run to
  int nt, mt;          // padded to tiles
  int count;           // matrices
  int first;           // the first one's number
  uint32_t from;       // the launch's first workgroup of this group
  int each, begin;     // where addresses are taken: workgroups of a matrix, the launch's first one
  int splits;          // of the sum over m
  int blocks;          // partial maxima
  int64_t base, stride;
  int64_t x, x2;       // X in its own order, and the product formed on the way
  int64_t sq;          // five n x n pairs: S, P, P S, and Q twice
  int64_t part, trace; // partial sums of S and of its trace, float32
  int64_t most, scale; // partial maxima; the factor on X
  bool tall;           // rows are the longer side
};
struct Groups {
  int count;
  Group g[kMaxGroups];
};
__device__ __forceinline__ uint8_t* square_of(const Group& g, uint8_t* own, int i) {
  return own + g.sq + (int64_t)i * g.nt * g.nt * 4;
}

__host__ __device__ inline int tri(int t) { return t * (t + 1) / 2; }

// Tile t of the upper triangle of nt x nt tiles: bands of eight rows, column by column, so that
// neighbours share both their rows and their columns (each XCD has an eighth of the tiles).
__device__ __forceinline__ void band_tile(int t, int nt, int& ti, int& tj) {
  constexpr int kBand = 8;
  int r0 = 0, high = min(nt, kBand);
  while (true) {   // a band has a triangle, then whole columns
    const int n = tri(high) + high * (nt - r0 - high);
    if (t < n) break;
    t -= n;
    r0 += high;
    high = min(nt - r0, kBand);
  }
  if (t < tri(high)) {
    int c = 0;
    while (t > c) t -= ++c;
    ti = r0 + t;
    tj = r0 + c;
  } else {
    t -= tri(high);
    ti = r0 + t % high;
    tj = r0 + high + t / high;
  }
}
// Tile t of the same, row by row.
__device__ __forceinline__ void tri_tile(int t, int nt, int& ti, int& tj) {
  int row = 0;
  while (t >= nt - row) {
    t -= nt - row;
    ++row;
  }
  ti = row;
  tj = row + t;
}

// Neighbouring tiles on one XCD: workgroups go round the eight of them.
__device__ __forceinline__ uint32_t by_xcd(uint32_t id, uint32_t total) {
  const uint32_t each = total / 8, more = total % 8, x = id % 8, i = id / 8;
  return x * each + min(x, more) + i;
}
__device__ __forceinline__ int group_of(const Groups& a, uint32_t id) {
  int g = 0;
  while (g + 1 < a.count && id >= a.g[g + 1].from) ++g;
  return __builtin_amdgcn_readfirstlane(g);
}

// How X's numbers are held: one half precision number, or two of them.
enum Form { kSingle, kPair };
typedef short short8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ f32x16 multiply(short8 a, short8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                0, 0);
}

// ---- the product loop ---------------------------------------------------------------------
__device__ __forceinline__ Rsrc rsrc(const void* base, int64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  const int n = __builtin_amdgcn_readfirstlane((int)min(bytes, (int64_t)0x7fffffff));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(((uint64_t)hi << 32) | lo),
                                           (short)0, n, 0x00020000);
}
// s_waitcnt vmcnt(N), the other counters left open.
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
// Waits until at most `later` stages of N copies each are under way; MOST: as many as there can be.
template <int N, int MOST>
__device__ __forceinline__ void wait_stages(int later) {
  if constexpr (MOST == 0) {
    wait_vm<0>();
  } else {
    if (later >= MOST) wait_vm<MOST * N>();
    else wait_stages<N, MOST - 1>(later);
  }
}
// LDS reads that are under way have arrived (lgkmcnt 0).
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void barrier_nofence() { asm volatile("s_barrier" ::: "memory"); }
__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 7); }

// One operand of a tile.  Straight: T rows of `ld` bytes, along which the sum runs.  Turned: the sum
// runs down rows of `ld` bytes, of which the tile has T columns, from p on.  A sum that is longer
// than the operand starts again at its first stage after `wrap`.
struct Side {
  const uint8_t* p;
  int64_t ld;
  int wrap;
};

typedef short short4_ __attribute__((ext_vector_type(4)));
// N fragments of 8 numbers along the sum, read from LDS rows that run across it: each 16 lanes of
// ds_read_b64_tr_b16 take four rows of 16 numbers, and each lane is left with a column's four.  at[i]
// is the lane's first address, LOW and HIGH the offsets of the first and the second four rows.  The
// wait stands in the same block: the compiler takes the registers as written at once.
template <int LOW, int HIGH>
__device__ __forceinline__ void read_turned(const uint32_t (&at)[1], short4_ (&x)[1][2]) {
  asm volatile(
      "ds_read_b64_tr_b16 %0, %2 offset:%3\n\t"
      "ds_read_b64_tr_b16 %1, %2 offset:%4\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0][0]), "=&v"(x[0][1])
      : "v"(at[0]), "n"(LOW), "n"(HIGH)
      : "memory");
}
template <int LOW, int HIGH>
__device__ __forceinline__ void read_turned(const uint32_t (&at)[2], short4_ (&x)[2][2]) {
  asm volatile(
      "ds_read_b64_tr_b16 %0, %4 offset:%6\n\t"
      "ds_read_b64_tr_b16 %1, %4 offset:%7\n\t"
      "ds_read_b64_tr_b16 %2, %5 offset:%6\n\t"
      "ds_read_b64_tr_b16 %3, %5 offset:%7\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0][0]), "=&v"(x[0][1]), "=&v"(x[1][0]), "=&v"(x[1][1])
      : "v"(at[0]), "v"(at[1]), "n"(LOW), "n"(HIGH)
      : "memory");
}
template <int LOW, int HIGH>
__device__ __forceinline__ void read_turned(const uint32_t (&at)[4], short4_ (&x)[4][2]) {
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8 offset:%12\n\t"
      "ds_read_b64_tr_b16 %1, %8 offset:%13\n\t"
      "ds_read_b64_tr_b16 %2, %9 offset:%12\n\t"
      "ds_read_b64_tr_b16 %3, %9 offset:%13\n\t"
      "ds_read_b64_tr_b16 %4, %10 offset:%12\n\t"
      "ds_read_b64_tr_b16 %5, %10 offset:%13\n\t"
      "ds_read_b64_tr_b16 %6, %11 offset:%12\n\t"
      "ds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0][0]), "=&v"(x[0][1]), "=&v"(x[1][0]), "=&v"(x[1][1]), "=&v"(x[2][0]), "=&v"(x[2][1]),
        "=&v"(x[3][0]), "=&v"(x[3][1])
      : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(LOW), "n"(HIGH)
      : "memory");
}

// A side's part of a stage in LDS: T rows of 128 bytes, or, turned, kDeep rows of T numbers (pairs:
// T hi and T lo in blocks).  16-byte chunks are swizzled by the row, so that reads meet no bank twice.
template <int T, Form F, bool TURNED, int WAVES>
struct Operand {
  static constexpr bool PAIR = F != kSingle;
  static constexpr int kB = T / 64;
  static constexpr int kBytes = T * kRowBytes;
  static constexpr int kCopies = kBytes / 1024 / WAVES;      // of a wave and stage, 1 KB each
  static constexpr int kDeep = PAIR ? 32 : 64;               // rows of a turned stage
  static constexpr int kAcross = TURNED ? T * (PAIR ? 4 : 2) : kRowBytes;   // bytes of a row in LDS
  static constexpr int kChunks = kAcross / 16;
  static constexpr int kReads = kB * (PAIR ? 2 : 1);         // fragments of a 16-deep step

  const uint8_t* p;
  int64_t ld;
  int wrap, k;
  Rsrc rs;
  uint32_t off[kCopies];
  uint32_t at[kReads];   // turned: the lane's pieces, from the side's start in a stage

  __device__ static __forceinline__ int swizzle(int row) {
    // turned: four rows of 16 columns (two chunks of each) are read at once
    return TURNED ? (kChunks >= 16 ? 4 : 2) * (row & 3) : swz(row);
  }
  __device__ __forceinline__ void start(const Side& s, int k0, int quarter) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    p = s.p;
    ld = s.ld;
    wrap = s.wrap;
    k = k0 % wrap;
    if (!TURNED) rs = rsrc(p, T * ld);
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      const int chunk = (wave + WAVES * q) * 64 + lane, row = chunk / kChunks;
      off[q] = (uint32_t)(row * ld) + (uint32_t)(((chunk % kChunks) ^ swizzle(row)) << 4);
    }
    if (TURNED) {
      const int g = lane >> 4, j = (lane >> 2) & 3, q = lane & 3;
      const int row = 8 * (g >> 1) + j;   // of the first four; (row & 3) is j in all of them
#pragma unroll
      for (int i = 0; i < kReads; ++i) {
        const int c = quarter * (T / 2) + 32 * (i % kB) + 16 * (g & 1) + 4 * q;
        const int chunk = PAIR ? (c >> 5) * 8 + (i / kB) * 4 + ((c & 31) >> 3) : c >> 3;
        at[i] = row * kAcross + ((chunk ^ swizzle(row)) << 4) + ((c >> 2) & 1) * 8;
      }
    }
  }
  __device__ __forceinline__ void issue(uint8_t* dst) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (TURNED) rs = rsrc(p + (int64_t)k * kDeep * ld, kDeep * ld);
#pragma unroll
    for (int q = 0; q < kCopies; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (__attribute__((address_space(3))) void*)(dst + (wave + WAVES * q) * 1024), 16,
          (int)off[q], TURNED ? 0 : k * kRowBytes, 0, 0);
    if (++k == wrap) k = 0;
  }
  // The hi (and lo) fragments of this wave's blocks for the 16-deep step u of a stage.
  template <int U>
  __device__ __forceinline__ void read(const uint8_t* src, int quarter, int first, short8 (&hi)[kB],
                                       short8 (&lo)[kB]) const {
    if constexpr (TURNED) {
      const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)src;
      uint32_t from[kReads];
      short4_ x[kReads][2];
#pragma unroll
      for (int i = 0; i < kReads; ++i) from[i] = base + at[i];
      read_turned<U * 16 * kAcross, (U * 16 + 4) * kAcross>(from, x);
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        hi[i] = __builtin_shufflevector(x[i][0], x[i][1], 0, 1, 2, 3, 4, 5, 6, 7);
        if constexpr (PAIR)
          lo[i] = __builtin_shufflevector(x[kB + i][0], x[kB + i][1], 0, 1, 2, 3, 4, 5, 6, 7);
      }
    } else {
      const int lane = threadIdx.x & 63, chunk = (first + U) * 2 + (lane >> 5);
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        const int row = quarter * (T / 2) + 32 * i + (lane & 31);
        const uint8_t* r = src + row * kRowBytes;
        hi[i] = *reinterpret_cast<const short8*>(r + ((chunk ^ swz(row)) << 4));
        if constexpr (PAIR) lo[i] = *reinterpret_cast<const short8*>(r + (((chunk + 4) ^ swz(row)) << 4));
      }
    }
  }
};

// A T x T tile of A B^T over the stages [k0, k0 + steps): each of four waves has a quarter, of eight
// waves two share one, each half of every stage (stage() adds them).  acc[i][j]
// are 32 x 32 blocks; in block (i, j) a lane has row lane % 32 of A's side and, as element
// 4 g + e, column 8 g + 4 (lane / 32) + e of B's.
//
// PAIR: three products of every hi + lo pair of fragments, 12 matrix instructions to 8 fragments
// read from LDS at T = 128 (single: 4 to 4).  RING stages are in flight, DEEP of them are taken between
// two barriers (two of four where T is 64: 300 x 4096 158 us in all, one at a time 165).
template <int T, int RING, Form F, int WAVES = 4, int DEEP = 1>
struct Product {
  static constexpr bool PAIR = F != kSingle;
  // The cross products are summed apart: a third of the additions to the large sum, whose roundings
  // the iteration raises (float32 results 1.1e-6 off instead of 1.4e-6 at 1031 x 517, 2.1e-6 instead
  // of 2.9e-6 at 300 x 300).  A tile of 128 has no registers for it.
  static constexpr bool kApart = F == kPair && T == 64;
  static constexpr int kB = T / 64;                       // blocks of a wave along a side
  static constexpr int kStage = 2 * T * kRowBytes;
  static constexpr int kCopies = kStage / 1024 / WAVES;   // of a wave and stage
  static constexpr int kHalves = WAVES / 4;               // waves that share a quarter
  static constexpr int kLds = RING * kStage;

  // TA, TB: that side is turned
  template <bool TA = false, bool TB = false>
  __device__ static __forceinline__ void run(uint8_t* sm, const Side& sa, const Side& sb, int k0,
                                             int steps, f32x16 (&acc)[kB][kB]) {
    static_assert(kHalves == 1 || (!TA && !TB), "halves of a stage are of straight sides");
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int quarter_a = wave & 1, quarter_b = (wave >> 1) & 1;
    Operand<T, F, TA, WAVES> a;
    Operand<T, F, TB, WAVES> b;
    a.start(sa, k0, quarter_a);
    b.start(sb, k0, quarter_b);
    auto issue = [&](int slot) {
      uint8_t* dst = sm + slot * kStage;
      a.issue(dst);
      b.issue(dst + a.kBytes);
    };
#pragma unroll
    for (int i = 0; i < kB; ++i)
#pragma unroll
      for (int j = 0; j < kB; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    f32x16 low[kApart ? kB : 1][kApart ? kB : 1];   // the cross products
    if (kApart) {
#pragma unroll
      for (int i = 0; i < kB; ++i)
#pragma unroll
        for (int j = 0; j < kB; ++j) low[kApart ? i : 0][kApart ? j : 0] = acc[i][j];
    }
    const int pre = min(RING, steps);
    for (int s = 0; s < pre; ++s) issue(s);
    constexpr int kSub = (PAIR ? 2 : 4) / kHalves;
    const int first = (wave >> 2) * kSub;   // the 16-deep steps of a stage that this wave takes
    int slot = 0;
    for (int s = 0; s < steps; s += DEEP) {
      // the stages have landed once only the copies of those behind them are in flight
      wait_stages<kCopies, RING - DEEP>(steps - DEEP - s);
      barrier_nofence();
#pragma unroll
      for (int d = 0; d < DEEP; ++d) {
        if (d > 0 && s + d >= steps) break;
        const uint8_t* src = sm + (slot + d) * kStage;
        auto step = [&](auto number) {
          constexpr int U = decltype(number)::value;
          short8 fa[kB], la[kB], fb[kB], lb[kB];
          a.template read<U>(src, quarter_a, first, fa, la);
          b.template read<U>(src + a.kBytes, quarter_b, first, fb, lb);
#pragma unroll
          for (int i = 0; i < kB; ++i)
#pragma unroll
            for (int j = 0; j < kB; ++j) {
              auto& c = acc[i][j];
              if constexpr (PAIR) {
                auto& l = kApart ? low[kApart ? i : 0][kApart ? j : 0] : c;
                l = multiply(fb[j], la[i], l);
                l = multiply(lb[j], fa[i], l);
              }
              c = multiply(fb[j], fa[i], c);
            }
        };
        step(std::integral_constant<int, 0>());
        if constexpr (kSub > 1) step(std::integral_constant<int, 1>());
        if constexpr (kSub > 2) {
          step(std::integral_constant<int, 2>());
          step(std::integral_constant<int, 3>());
        }
      }
      // every wave has read the slots, and not only asked for them, before they are filled again
      wait_lds();
      barrier_nofence();
#pragma unroll
      for (int d = 0; d < DEEP; ++d)
        if (s + d + RING < steps) issue(slot + d);
      slot += DEEP;
      if (slot == RING) slot = 0;
    }
    if (kApart) {
#pragma unroll
      for (int i = 0; i < kB; ++i)
#pragma unroll
        for (int j = 0; j < kB; ++j) acc[i][j] += low[kApart ? i : 0][kApart ? j : 0];
    }
  }

  // The tile in LDS, for results that leave in whole rows (or columns) of it: a lane's four columns
  // of 32 different rows would be 8 bytes here and there.  Groups of four columns are swizzled by
  // the row, so that rows and columns are read without bank conflicts.
  __device__ static __forceinline__ float* at(float* tile, int r, int c) {
    return tile + r * T + (((c >> 2) ^ ((r ^ (r >> 3)) & (T / 4 - 1))) << 2) + (c & 3);
  }
  __device__ static __forceinline__ float* stage(uint8_t* sm, const f32x16 (&acc)[kB][kB]) {
    static_assert(T * T * 4 <= kLds, "the tile fits where the stages were");
    float* tile = reinterpret_cast<float*>(sm);
#pragma unroll
    for (int half = 0; half < kHalves; ++half) {
      if (kHalves == 1 || (int)threadIdx.x / 256 == half)
        each(acc, [&](int r, int c, f32x4 v) {
          f32x4* p = reinterpret_cast<f32x4*>(at(tile, r, c));
          *p = half ? *p + v : v;
        });
      __syncthreads();
    }
    return tile;
  }
  // Eight columns of a row, and eight rows of a column.
  __device__ static __forceinline__ void row8(float* tile, int r, int c, float* v) {
#pragma unroll
    for (int q = 0; q < 8; q += 4) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(at(tile, r, c + q));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[q + e] = x[e];
    }
  }
  __device__ static __forceinline__ void column8(float* tile, int r, int c, float* v) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = *at(tile, r + q, c);
  }
  // Calls fn(line, first of eight) for all of the tile's lines; numbered: fn(which of this thread's, ..).
  static constexpr int kLines = T * T / 8 / (WAVES * 64);
  template <typename Fn>
  __device__ static __forceinline__ void numbered(Fn fn) {
#pragma unroll
    for (int i = 0; i < kLines; ++i) {
      const int x = i * WAVES * 64 + threadIdx.x;
      fn(i, x / (T / 8), x % (T / 8) * 8);
    }
  }
  template <typename Fn>
  __device__ static __forceinline__ void lines(Fn fn) {
    numbered([&](int, int r, int c) { fn(r, c); });
  }
  // Calls fn(row, column, values of four columns) for every group of four that this lane has.
  template <typename Fn>
  __device__ static __forceinline__ void each(const f32x16 (&acc)[kB][kB], Fn fn) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < kB; ++i)
#pragma unroll
      for (int j = 0; j < kB; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          fn((wave & 1) * (T / 2) + 32 * i + (lane & 31),
             ((wave >> 1) & 1) * (T / 2) + 32 * j + 8 * g + 4 * (lane >> 5),
             f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                   acc[i][j][4 * g + 3]});
  }
};

// ---- pairs ----------------------------------------------------------------------------------
__device__ __forceinline__ int64_t pair_at(int64_t k) { return (k >> 5) * 64 + (k & 31); }

// v is rounded to float32 first, in a register: a product that the compiler rounds to hi in one
// step (v_fma_mixlo_f16) and to float32 for lo has another hi in one of 4000 cases.
__device__ __forceinline__ void split(float v, f16& hi, f16& lo) {
  asm("" : "+v"(v));
  hi = (f16)v;
  lo = (f16)(v - (float)hi);
}
// Columns [k, k + N) of a pair row; of a flat one, whose lo begin at `lo`.
template <int N>
__device__ __forceinline__ void store_pair(f16* row, int64_t k, const float* v, int64_t lo = 0) {
  typedef f16 V __attribute__((ext_vector_type(N)));
  V h, l;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    f16 a, b;
    split(v[e], a, b);
    h[e] = a;
    l[e] = b;
  }
  f16* p = row + (lo ? k : pair_at(k));
  *reinterpret_cast<V*>(p) = h;
  *reinterpret_cast<V*>(p + (lo ? lo : kPairBlock)) = l;
}
__device__ __forceinline__ void load_pair8(const f16* row, int64_t k, float* v) {
  const f16* p = row + pair_at(k);
  const f16x8 h = *reinterpret_cast<const f16x8*>(p);
  const f16x8 l = *reinterpret_cast<const f16x8*>(p + kPairBlock);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)h[e] + (float)l[e];
}

// ---- X into half precision --------------------------------------------------------------------
// Where a matrix's elements come from.  MOMENT: u = mu m + (1 - mu) g of the gradient in `x` and
// the momentum (already moved on where `moved`), or the momentum itself without nesterov.
struct Source {
  const void* x;
  float* moment;
};
struct Sources {
  Groups groups;
  int first;                       // number of the launch's first matrix
  Source s[kMaxMatrices];
  float mu, nu;                    // momentum's factor, 1 - that
  int nesterov;
};

// Which matrix a workgroup of a launch with addresses works on.
struct Where {
  const Group& g;
  int slot;      // of the launch's addresses
  int piece;     // of the matrix's workgroups
  uint8_t* own;
};
__device__ __forceinline__ Where where(const Groups& a, int first, uint32_t id, uint8_t* ws) {
  const Group& g = a.g[group_of(a, id)];
  const int u = (int)(id - g.from) / g.each, matrix = g.begin + u;
  return {g, __builtin_amdgcn_readfirstlane(matrix - first), (int)(id - g.from) - u * g.each,
          ws + g.base + (int64_t)(matrix - g.first) * g.stride};
}
__device__ __forceinline__ float moved(float m, float g, float mu, float nu) {
  return fmaf(mu, m, nu * g);
}
__device__ __forceinline__ float update_of(float m, float g, const Sources& a) {
  return a.nesterov ? fmaf(a.mu, m, a.nu * g) : m;
}

constexpr int kVec = 8;

template <bool BF>
__device__ __forceinline__ void load8(const void* p, int64_t i, int64_t n, float* v) {
  using E = Elem<BF>;
  const typename E::T* x = reinterpret_cast<const typename E::T*>(p);
#pragma unroll
  for (int q = 0; q < kVec; q += E::kN) load_part<BF>(x, i + q, n, 0.f, v + q);
}

// The largest magnitude of a matrix's part, as bits (NaN above infinity above numbers), and the
// momentum moved on: one pass over gradient and momentum, bound by memory.
template <bool BF, bool MOMENT>
__global__ __launch_bounds__(kThreads) void dora_orthogonal_most(const Sources a, uint8_t* ws) {
  __shared__ uint32_t lds[kThreads / 64];
  const Where at = where(a.groups, a.first, blockIdx.x, ws);
  const Group& g = at.g;
  const int64_t n = (int64_t)g.n * g.m;
  const int block = at.piece;
  const Source s = a.s[at.slot];
  uint32_t most = 0;
  for (int64_t i = ((int64_t)block * kThreads + threadIdx.x) * kVec; i < n;
       i += (int64_t)g.blocks * kThreads * kVec) {
    float v[kVec];
    load8<BF>(s.x, i, n, v);
    if (MOMENT) {
      float m[kVec];
      load8<false>(s.moment, i, n, m);
#pragma unroll
      for (int q = 0; q < kVec; ++q) {
        m[q] = moved(m[q], v[q], a.mu, a.nu);
        v[q] = update_of(m[q], v[q], a);
      }
      store_part<false>(s.moment, i, n, m);
      store_part<false>(s.moment, i + 4, n, m + 4);
    }
#pragma unroll
    for (int q = 0; q < kVec; ++q) most = max(most, __float_as_uint(v[q]) & 0x7fffffffu);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) most = max(most, (uint32_t)__shfl_xor((int)most, off, 64));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) most = max(most, lds[w]);
    reinterpret_cast<uint32_t*>(at.own + g.most)[block] = most;
  }
}

// The power of two that takes a matrix's largest magnitude to [2^14, 2^15): half precision holds
// 2^16 - 32 at most and whole steps of 2^-24.  0 for a matrix of zeros, infinities or NaN (whose
// results are NaN throughout).
__device__ __forceinline__ uint32_t most_of(const uint32_t* most, int blocks) {   // a thread's part
  uint32_t v = 0;
  for (int i = threadIdx.x; i < blocks; i += kThreads) v = max(v, most[i]);
  return v;
}
__device__ __forceinline__ int exponent_of(uint32_t v, uint32_t* lds) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 64));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) v = max(v, lds[w]);
  if (v == 0 || v >= 0x7f800000u) return 0;
  const int e = v >> 23 ? (int)(v >> 23) - 127 : 31 - __builtin_clz(v) - 149;
  return 14 - e;
}

// The padded matrix as half precision numbers, zeros where the matrix ends: a thread takes eight
// columns.  Memory bounds it: 2 to 6 bytes an element are read, 2 or 4 written.
constexpr int kPiece = 4096;   // elements of a workgroup
template <bool BF, bool MOMENT, Form F>
__global__ __launch_bounds__(kThreads) void dora_orthogonal_halves(const Sources a, uint8_t* ws) {
  constexpr bool PAIR = F == kPair;
  __shared__ uint32_t lds[kThreads / 64];
  const Where here = where(a.groups, a.first, blockIdx.x, ws);
  const Group& g = here.g;
  uint8_t* own = here.own;
  const int rows = g.tall ? g.m : g.n, cols = g.tall ? g.n : g.m;
  const int pcols = g.tall ? g.nt : g.mt;
  const int64_t all = (int64_t)g.nt * g.mt;
  const int e = exponent_of(most_of(reinterpret_cast<const uint32_t*>(own + g.most), g.blocks), lds);
  const Source s = a.s[here.slot];
  f16* out = reinterpret_cast<f16*>(own + g.x);
  const int64_t first = (int64_t)here.piece * kPiece, row0 = first / pcols;
  const uint32_t col0 = (uint32_t)(first - row0 * pcols);
#pragma unroll
  for (int i = 0; i < kPiece / kVec / kThreads; ++i) {
    const uint32_t on = col0 + (i * kThreads + threadIdx.x) * kVec, down = on / (uint32_t)pcols;
    const int64_t r = row0 + down, at = first + (on - col0);
    const int c = (int)(on - down * (uint32_t)pcols);
    if (at >= all) break;
    float v[kVec] = {};
    if (r < rows && c < cols) {
      const int64_t from = r * cols + c, stop = (r + 1) * cols;   // the row's end: zeros behind it
      load8<BF>(s.x, from, stop, v);
      if (MOMENT) {
        float m[kVec];
        load8<false>(s.moment, from, stop, m);
#pragma unroll
        for (int q = 0; q < kVec; ++q) v[q] = update_of(m[q], v[q], a);
      }
    }
    f16x8 h, l;
#pragma unroll
    for (int q = 0; q < kVec; ++q) {
      f16 x, y;
      split(ldexpf(v[q], e), x, y);
      h[q] = x;
      l[q] = y;
    }
    f16* p = out + (PAIR ? r * pcols * 2 + pair_at(c) : at);
    *reinterpret_cast<f16x8*>(p) = h;
    if (PAIR) *reinterpret_cast<f16x8*>(p + kPairBlock) = l;
  }
}

// ---- n x n products ---------------------------------------------------------------------------
// Partial sums of S = X X^T over a part of m, float32.
template <int T, int RING, Form F>
__global__ __launch_bounds__(kThreads) void dora_orthogonal_gram(const Groups a, uint32_t total,
                                                                 bool second, uint8_t* ws) {
  using P = Product<T, RING, F, 4, T == 64 ? 2 : 1>;
  constexpr bool PAIR = P::PAIR;
  __shared__ __attribute__((aligned(1024))) uint8_t sm[P::kLds];
  const uint32_t id = by_xcd(blockIdx.x, total);
  const Group& g = a.g[group_of(a, id)];
  const int nt = (g.n + T - 1) / T, tiles = tri(nt);
  int rest = (int)(id - g.from);
  const int split = rest % g.splits;
  rest /= g.splits;
  const int t = rest % tiles, u = rest / tiles;
  int ti, tj;
  tri_tile(t, nt, ti, tj);
  uint8_t* own = ws + g.base + (int64_t)u * g.stride;
  constexpr int kSize = PAIR ? 4 : 2;   // bytes of a number
  const int64_t ld = (int64_t)(g.tall ? g.nt : g.mt) * kSize;
  const int stages = (g.m + 63) / 64 * (PAIR ? 2 : 1);
  const int k0 = (int)((int64_t)stages * split / g.splits);
  const int k1 = (int)((int64_t)stages * (split + 1) / g.splits);
  const uint8_t* x = own + (second ? g.x2 : g.x);
  f32x16 acc[P::kB][P::kB];
  if (g.tall)
    P::template run<true, true>(sm, Side{x + ti * T * kSize, ld, stages},
                                Side{x + tj * T * kSize, ld, stages}, k0, k1 - k0, acc);
  else
    P::run(sm, Side{x + ti * T * ld, ld, stages}, Side{x + tj * T * ld, ld, stages}, k0, k1 - k0, acc);
  float* out = reinterpret_cast<float*>(own + g.part) + ((int64_t)t * g.splits + split) * T * T;
  P::each(acc, [&](int i, int j, const f32x4& v) {
    *reinterpret_cast<f32x4*>(out + i * T + j) = v;
  });
  if (ti != tj) return;
  float sum = 0.f;
  P::each(acc, [&](int i, int j, const f32x4& v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += i == j + e ? v[e] : 0.f;
  });
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0)
    reinterpret_cast<float*>(own + g.trace)[(ti * g.splits + split) * kWaves + threadIdx.x / 64] = sum;
}

// ---- n <= 64: S while X is written or taken further -----------------------------------------------
// A block of 64 of the longer side is all that S's sum needs of it, and fits a workgroup's LDS.

// A wave's quarter of S, 32 x 32, summed over blocks in LDS (`TURNED`: their rows run across the sum).
template <Form F, bool TURNED>
struct Sums {
  using Side64 = Operand<64, F, TURNED, kWaves>;
  static constexpr bool PAIR = F != kSingle;
  static constexpr int kStages = PAIR ? 2 : 1, kBytes = Side64::kBytes;   // of a block
  static constexpr int kBlock = kStages * kBytes;
  Side64 a, b;
  f32x16 acc, low;

  __device__ __forceinline__ Sums() {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Side none = {nullptr, 0, 1};
    a.start(none, 0, wave & 1);
    b.start(none, 0, wave >> 1);
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = low[e] = 0.f;
  }
  // Where eight columns of a row of X begin in a block; a pair's lo lie kLo chunks on.
  __device__ static __forceinline__ uint8_t* at(uint8_t* block, int row, int c, int lo) {
    if constexpr (TURNED) {
      const int chunk = PAIR ? (c >> 5) * 8 + ((c & 31) >> 3) + lo : c >> 3;
      return block + row * Side64::kAcross + ((chunk ^ Side64::swizzle(row)) << 4);
    } else {
      const int chunk = PAIR ? ((c & 31) >> 3) + lo : c >> 3;
      return block + (PAIR ? (c >> 5) * kBytes : 0) + row * kRowBytes + ((chunk ^ swz(row)) << 4);
    }
  }
  __device__ __forceinline__ void add(const uint8_t* block) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    auto step = [&](const uint8_t* src, auto number) {
      constexpr int U = decltype(number)::value;
      short8 fa[1], la[1], fb[1], lb[1];
      a.template read<U>(src, wave & 1, 0, fa, la);
      b.template read<U>(src, wave >> 1, 0, fb, lb);
      if constexpr (PAIR) {
        low = multiply(fb[0], la[0], low);
        low = multiply(lb[0], fa[0], low);
      }
      acc = multiply(fb[0], fa[0], acc);
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
      step(block + s * kBytes, std::integral_constant<int, 0>());
      step(block + s * kBytes, std::integral_constant<int, 1>());
    }
    if constexpr (!PAIR) {
      step(block, std::integral_constant<int, 2>());
      step(block, std::integral_constant<int, 3>());
    }
  }
  // The partial sums and this wave's part of their trace, as dora_orthogonal_gram leaves them.
  __device__ __forceinline__ void give(const Group& g, uint8_t* own, int split) {
    using P = Product<64, 4, F>;
    const f32x16 all[1][1] = {{acc + low}};
    float* out = reinterpret_cast<float*>(own + g.part) + (int64_t)split * 64 * 64;
    float sum = 0.f;
    P::each(all, [&](int i, int j, const f32x4& v) {
      *reinterpret_cast<f32x4*>(out + i * 64 + j) = v;
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += i == j + e ? v[e] : 0.f;
    });
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0)
      reinterpret_cast<float*>(own + g.trace)[split * kWaves + threadIdx.x / 64] = sum;
  }
};

// X as halves (see dora_orthogonal_halves) and the sums of S over it in one pass: X is written, but
// not read again for S.  The numbers of the next block are under way while this one is multiplied.
// Memory bounds it: 56 layers' 29M elements, 10 bytes each, take 68 us (4.3 TB/s), where the two
// kernels that n > 64 has took 67 and 42.  Three workgroups to a CU, for which one variant spills two
// registers (two to a CU: 72 us).
template <bool BF, bool MOMENT, Form F>
__global__ __launch_bounds__(kThreads, 3) void dora_orthogonal_first(const Sources a, uint8_t* ws) {
  constexpr bool PAIR = F == kPair;
  constexpr int kBlock = Sums<F, false>::kBlock, kMine = 64 * 64 / kVec / kThreads;
  __shared__ __attribute__((aligned(1024))) uint8_t sm[2][kBlock];
  __shared__ uint32_t lds[kThreads / 64];
  const Where here = where(a.groups, a.first, blockIdx.x, ws);
  const Group& g = here.g;
  const Source s = a.s[here.slot];
  const int e = exponent_of(most_of(reinterpret_cast<const uint32_t*>(here.own + g.most), g.blocks), lds);
  const int rows = g.tall ? g.m : g.n, cols = g.tall ? g.n : g.m, pcols = g.tall ? g.nt : g.mt;
  const int blocks = (g.m + 63) / 64;
  const int k0 = (int)((int64_t)blocks * here.piece / g.splits);
  const int k1 = (int)((int64_t)blocks * (here.piece + 1) / g.splits);
  f16* out = reinterpret_cast<f16*>(here.own + g.x);
  auto run = [&](auto tall) {
    constexpr bool TALL = decltype(tall)::value;
    Sums<F, TALL> sums;
    float v[kMine][kVec], m[MOMENT ? kMine : 1][kVec];
    auto place = [&](int k, int i, int& r, int& c, int64_t& r_all, int64_t& c_all) {
      r = (i * kThreads + (int)threadIdx.x) / 8;
      c = (int)threadIdx.x % 8 * kVec;
      r_all = r + (TALL ? (int64_t)k * 64 : 0);
      c_all = c + (TALL ? 0 : (int64_t)k * 64);
      return r_all < rows && c_all < cols;
    };
    auto load = [&](int k) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        int r, c;
        int64_t ra, ca;
#pragma unroll
        for (int q = 0; q < kVec; ++q) v[i][q] = m[MOMENT ? i : 0][q] = 0.f;
        if (!place(k, i, r, c, ra, ca)) continue;
        load8<BF>(s.x, ra * cols + ca, (ra + 1) * cols, v[i]);
        if (MOMENT) load8<false>(s.moment, ra * cols + ca, (ra + 1) * cols, m[MOMENT ? i : 0]);
      }
    };
    load(k0);
    for (int k = k0; k < k1; ++k) {
      uint8_t* block = sm[(k - k0) & 1];
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        int r, c;
        int64_t ra, ca;
        place(k, i, r, c, ra, ca);
        if (MOMENT) {
#pragma unroll
          for (int q = 0; q < kVec; ++q) v[i][q] = update_of(m[MOMENT ? i : 0][q], v[i][q], a);
        }
        f16x8 h, l;
#pragma unroll
        for (int q = 0; q < kVec; ++q) {
          // (behind a row's end are zeros, and update_of of the zeros of gradient and momentum)
          f16 x, y;
          split(ldexpf(v[i][q], e), x, y);
          h[q] = x;
          l[q] = y;
        }
        f16* to = out + (PAIR ? ra * pcols * 2 + pair_at(ca) : ra * pcols + ca);
        *reinterpret_cast<f16x8*>(to) = h;
        *reinterpret_cast<f16x8*>(sums.at(block, r, c, 0)) = h;
        if (PAIR) {
          *reinterpret_cast<f16x8*>(to + kPairBlock) = l;
          *reinterpret_cast<f16x8*>(sums.at(block, r, c, 4)) = l;
        }
      }
      if (k + 1 < k1) load(k + 1);
      wait_lds();
      barrier_nofence();
      sums.add(block);   // (the other block is written next, this one behind another barrier)
      wait_lds();
    }
    sums.give(g, here.own, here.piece);
  };
  if (g.tall) run(std::true_type());
  else run(std::false_type());
}

// Y = Q_k .. Q_1 X for a block of 64 of X's longer side, with each product rounded to a pair: what
// was formed from it before is the same to the bit, whoever forms it again.  (One product with the Q
// of all steps in its place would not be what S was summed from: a matrix of rank 2 came out 2e-4 off
// instead of 2e-5.)
constexpr int kMostQ = 3;
struct Turns {
  float unit[kMostQ];   // of each product; the first one's times X's own
};
constexpr int kHalfBlock = 64 * kRowBytes, kPairs = 2 * kHalfBlock;   // bytes of a block's half, and of it

// 32 rows of Q, 16 columns each.
struct Rows {
  short8 h[4], l[4];
  __device__ __forceinline__ void load(const Group& g, uint8_t* own, int number, int first) {
    const int lane = threadIdx.x & 63;
    const f16* q = reinterpret_cast<const f16*>(square_of(g, own, number)) + (first + (lane & 31)) * 128;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const f16* p = q + pair_at(u * 16 + (lane >> 5) * 8);
      h[u] = *reinterpret_cast<const short8*>(p);
      l[u] = *reinterpret_cast<const short8*>(p + kPairBlock);
    }
  }
};
// A quarter of Q times a block in LDS: a lane has a row of Q and, as element 4 g + e, column 8 g + 4
// (lane / 32) + e of the block; ACROSS: a column of the block and these rows of Q.
template <bool ACROSS, bool TURNED>
__device__ __forceinline__ f32x16 quarter_of(const Rows& q, const Operand<64, kPair, TURNED, kWaves>& x,
                                             const uint8_t* block, int quarter) {
  f32x16 acc, low;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = low[e] = 0.f;
  auto step = [&](auto number) {
    constexpr int U = decltype(number)::value;
    short8 h[1], l[1];
    x.template read<U % 2>(block + U / 2 * kHalfBlock, quarter, 0, h, l);
    low = ACROSS ? multiply(q.l[U], h[0], low) : multiply(h[0], q.l[U], low);
    low = ACROSS ? multiply(q.h[U], l[0], low) : multiply(l[0], q.h[U], low);
    acc = ACROSS ? multiply(q.h[U], h[0], acc) : multiply(h[0], q.h[U], acc);
  };
  step(std::integral_constant<int, 0>());
  step(std::integral_constant<int, 1>());
  step(std::integral_constant<int, 2>());
  step(std::integral_constant<int, 3>());
  return acc + low;
}
// Puts a quarter of Y into a block: its sum is to run down the rows (TURNED) or along them.
template <bool TURNED>
__device__ __forceinline__ void keep_quarter(uint8_t* block, const f32x16& acc, float f, int qa, int qb) {
  const int lane = threadIdx.x & 63, i = qa * 32 + (lane & 31);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    f16x4 h, l;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f16 hi, lo;
      split(acc[4 * c + e] * f, hi, lo);
      h[e] = hi;
      l[e] = lo;
    }
    const int at = qb * 32 + c * 8;
    *reinterpret_cast<f16x4*>(Sums<kPair, TURNED>::at(block, i, at, 0) + (lane >> 5) * 8) = h;
    *reinterpret_cast<f16x4*>(Sums<kPair, TURNED>::at(block, i, at, 4) + (lane >> 5) * 8) = l;
  }
}
// Copies block k of X, two stages of 32 of n.
template <bool TALL>
__device__ __forceinline__ void issue_block(Operand<64, kPair, !TALL, kWaves>& x, const uint8_t* from,
                                            int64_t ld, int64_t k, uint8_t* to) {
  x.p = from + k * 64 * (TALL ? ld : 4);
  if (TALL) x.rs = rsrc(x.p, 64 * ld);
  x.issue(to);
  x.issue(to + kHalfBlock);
}

// S anew after QS segments: the sums of Y Y^T, in one pass over X; Y is not kept.  56 layers' 29M
// elements take 39 us, of which reading X alone is 27; a product that is kept and sums of it (as n > 64
// has) took 56 and 42.  48 KB of LDS put three workgroups on a CU (a ring of three blocks, two
// workgroups: 61 us).
template <int QS>
__global__ __launch_bounds__(kThreads) void dora_orthogonal_fold(const Groups a, uint32_t total,
                                                                 const Turns turns, uint8_t* ws) {
  constexpr int kRing = 2;   // (48 KB with `made`: three workgroups to a CU)
  __shared__ __attribute__((aligned(1024))) uint8_t sm[kRing][kPairs];
  __shared__ __attribute__((aligned(1024))) uint8_t made[QS][kPairs];
  const uint32_t id = by_xcd(blockIdx.x, total);
  const Group& g = a.g[group_of(a, id)];
  const int rest = (int)(id - g.from), part = rest % g.splits;
  uint8_t* own = ws + g.base + (int64_t)(rest / g.splits) * g.stride;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), qa = wave & 1, qb = wave >> 1;
  const int64_t ld = (int64_t)(g.tall ? g.nt : g.mt) * 4;
  const int blocks = (g.m + 63) / 64;
  const int k0 = (int)((int64_t)blocks * part / g.splits);
  const int k1 = (int)((int64_t)blocks * (part + 1) / g.splits);
  const float f = *reinterpret_cast<const float*>(own + g.scale) * turns.unit[0];
  Rows q[QS];
#pragma unroll
  for (int i = 0; i < QS; ++i) q[i].load(g, own, i, qa * 32);
  auto run = [&](auto tall) {
    constexpr bool TALL = decltype(tall)::value;
    Sums<kPair, false> sums;
    Operand<64, kPair, !TALL, kWaves> x;
    x.start(Side{own + g.x, ld, 2}, 0, qb);
    Operand<64, kPair, true, kWaves> y;   // Y of all but the last segment
    y.start(Side{nullptr, 0, 1}, 0, qb);
    constexpr int kCopies = 2 * x.kCopies;
    for (int k = k0; k < min(k0 + kRing, k1); ++k) issue_block<TALL>(x, own + g.x, ld, k, sm[(k - k0) & 1]);
    for (int k = k0; k < k1; ++k) {
      if (k + 1 < k1) wait_vm<kCopies>();
      else wait_vm<0>();
      barrier_nofence();   // also: Y of the block before has been read
      uint8_t* src = sm[(k - k0) & 1];
      keep_quarter<QS == 2>(made[0], quarter_of<false>(q[0], x, src, qb), f, qa, qb);
      wait_lds();
      barrier_nofence();   // Y is there, and the block of X has been read
      if (k + kRing < k1) issue_block<TALL>(x, own + g.x, ld, k + kRing, src);
      if (QS == 2) {
        keep_quarter<false>(made[QS - 1], quarter_of<false>(q[QS - 1], y, made[0], qb), turns.unit[1], qa, qb);
        wait_lds();
        barrier_nofence();
      }
      sums.add(made[QS - 1]);
      wait_lds();
    }
    sums.give(g, own, part);
  };
  if (g.tall) run(std::true_type());
  else run(std::false_type());
}

// What turns X' X'^T into the first S: X' is X times the power of two that its largest element asks for.
struct Unit {
  float unit;   // the factor on X' where it is known, else 0
  float eps;
};
__device__ __forceinline__ float norm_factor(float trace, const Unit& u, uint32_t most, uint32_t* lds) {
  return 1.f / (sqrtf(trace) + ldexpf(u.eps, exponent_of(most, lds)));
}

// Adds S's partial sums in order, and makes it a pair.  `unit` 0: X is normalised here: the factor
// 1 / (|X| + eps) comes from the trace, which every workgroup adds up for itself in the same order
// (four numbers for each split of a tile).  Otherwise the factor is `unit`.
template <int T>
__global__ __launch_bounds__(kThreads) void dora_orthogonal_gather(const Groups a, const Unit unit,
                                                                   float to, uint8_t* ws) {
  constexpr int kE = 32, kSide = T / kE;
  __shared__ float tile[kE][kE + 1];
  __shared__ float lds[kThreads / 64];
  __shared__ uint32_t lds_most[kThreads / 64];
  const uint32_t id = blockIdx.x;
  const Group& g = a.g[group_of(a, id)];
  const int nt = (g.n + T - 1) / T, tiles = tri(nt);
  int rest = (int)(id - g.from);
  const int piece = rest % (kSide * kSide);
  rest /= kSide * kSide;
  const int t = rest % tiles, u = rest / tiles;
  int ti, tj;
  tri_tile(t, nt, ti, tj);
  uint8_t* own = ws + g.base + (int64_t)u * g.stride;
  const float* part = reinterpret_cast<const float*>(own + g.part);
  float r = unit.unit;
  if (r == 0.f) {
    float sum[1] = {0.f};
    const float* d = reinterpret_cast<const float*>(own + g.trace);
    for (int i = threadIdx.x; i < nt * g.splits * kWaves; i += kThreads) sum[0] += d[i];
    block_sum<kThreads / 64, 1>(sum, lds);
    r = norm_factor(sum[0], unit, most_of(reinterpret_cast<const uint32_t*>(own + g.most), g.blocks), lds_most);
  }
  if (piece == 0 && t == 0 && threadIdx.x == 0) *reinterpret_cast<float*>(own + g.scale) = r;
  const int pi = piece / kSide * kE, pj = piece % kSide * kE;
  if (ti == tj && pj < pi) return;   // (the same for the whole workgroup)
  const int i = threadIdx.x / 8, j = threadIdx.x % 8 * 4;
  const float* p = part + (int64_t)t * g.splits * T * T + (pi + i) * T + pj + j;
  double x[4] = {};
  for (int s = 0; s < g.splits; ++s) {
    const f32x4 d = *reinterpret_cast<const f32x4*>(p + (int64_t)s * T * T);
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] += (double)d[q];
  }
  float v[4], w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = (float)x[q] * r * r * to;
#pragma unroll
  for (int q = 0; q < 4; ++q) tile[i][j + q] = v[q];
  __syncthreads();
  const bool diagonal = ti == tj && pi == pj;
  if (diagonal) {   // the upper half's values on both sides
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (j + q < i) v[q] = tile[j + q][i];
  }
  f16* s = reinterpret_cast<f16*>(square_of(g, own, 0));
  const int64_t ld = 2 * (int64_t)g.nt;
  const int64_t row = (int64_t)ti * T + pi, col = (int64_t)tj * T + pj;
  store_pair<4>(s + (row + i) * ld, col + j, v);
  if (diagonal) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) w[q] = tile[j + q][i];
  store_pair<4>(s + (col + i) * ld, row + j, w);
}

// A symmetric product of two n x n pairs, or of two such products of one launch (`both`).
//   POLY: out = alpha (left right) + beta left + gamma 1, left and right both S
//   otherwise out = alpha (left right)
// `form`: as X's form wants Q: kSingle: all hi of a row, then all lo.
struct Square {
  int left, right, out;      // of sq
  float alpha, beta, gamma;
  int form;
};
struct Squares {
  Groups groups;
  uint32_t total, half;      // workgroups; where the second product starts (total: there is none)
  Square q[2];
};
template <int T, int RING, int WAVES, int DEEP, bool POLY>
__global__ __launch_bounds__(WAVES * 64) void dora_orthogonal_square(const Squares a, uint8_t* ws) {
  using P = Product<T, RING, kPair, WAVES, DEEP>;
  __shared__ __attribute__((aligned(1024))) uint8_t sm[P::kLds];
  uint32_t id = by_xcd(blockIdx.x, a.total);
  const Square& q = a.q[id >= a.half ? 1 : 0];
  if (id >= a.half) id -= a.half;
  const Group& g = a.groups.g[group_of(a.groups, id)];
  const int nt = (g.n + T - 1) / T, tiles = tri(nt);
  const int rest = (int)(id - g.from);
  const int t = rest % tiles, u = rest / tiles;
  int ti, tj;
  band_tile(t, nt, ti, tj);
  uint8_t* own = ws + g.base + (int64_t)u * g.stride;
  const int64_t ld = (int64_t)g.nt * 4, le = ld / 2;
  const int stages = g.ne / kPairBlock;
  const uint8_t* left = square_of(g, own, q.left);
  const int64_t i0 = (int64_t)ti * T, j0 = (int64_t)tj * T;
  f32x16 acc[P::kB][P::kB];
  P::run(sm, Side{left + i0 * ld, ld, stages}, Side{square_of(g, own, q.right) + j0 * ld, ld, stages}, 0,
         stages, acc);
  float* tile = P::stage(sm, acc);
  f16* out = reinterpret_cast<f16*>(square_of(g, own, q.out));
  // columns [j, j + 8) of row i
  auto put = [&](int64_t i, int64_t j, float* v) {
    if (j >= g.ne) return;   // padding that nothing reads (and where a flat row's lo lie)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= q.alpha;
    if (POLY) {
      float s[8];
      load_pair8(reinterpret_cast<const f16*>(left) + i * le, j, s);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = fmaf(q.beta, s[e], v[e]);
        if (i == j + e && i < g.n) v[e] += q.gamma;
      }
    }
    store_pair<8>(out + i * le, j, v, q.form == kSingle ? g.ne : 0);
  };
  P::lines([&](int r, int c) {
    float v[8];
    P::row8(tile, r, c, v);
    if (ti == tj && c < r) {   // below the diagonal what is above it, so that it stays symmetric
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < r) v[e] = *P::at(tile, c + e, r);
    }
    put(i0 + r, j0 + c, v);
  });
  if (ti == tj) return;
  P::lines([&](int c, int r) {
    float v[8];
    P::column8(tile, r, c, v);
    put(j0 + c, i0 + r, v);
  });
}

// All of a segment's n x n products for n <= 64: one workgroup a matrix, with S, P, P S and Q in
// LDS.  A product is 12 matrix instructions of each of four waves; waiting for LDS and for each other
// bounds it (a step of three or four products 2.3 us, the sums' gathering 6), so that all reads of a
// phase stand before its writes, and P's rows and S's stay in registers for the products that share
// them.  Five steps take 19 us where as many launches take 75.
struct Chain {
  Groups groups;
  int steps;
  Unit unit;                           // as dora_orthogonal_gather's
  float to;
  int form;                            // X's, which says how Q is wanted
  int q;                               // where it is put
  bool scale;                          // X's factor is put down
  float step[kMaxSteps][6];            // factors of S S, S and 1; of P S, P Q and P (P S)
};
__global__ __launch_bounds__(kThreads) void dora_orthogonal_chain(const Chain a, uint8_t* ws) {
  constexpr int kN = 64, kLd = kN * 4;   // bytes of a pair row: 16 chunks, swizzled by the row
  __shared__ __attribute__((aligned(1024))) uint8_t sm[5][kN * kLd];
  __shared__ float lds[kThreads / 64];
  __shared__ uint32_t lds_most[kThreads / 64];
  __shared__ float steps[kMaxSteps * 6];
  const Group& g = a.groups.g[group_of(a.groups, blockIdx.x)];
  uint8_t* own = ws + g.base + (int64_t)(blockIdx.x - g.from) * g.stride;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = g.n;
  // all at once: a step that asks the kernel's arguments for its own waits 3000 cycles for them
  if ((int)threadIdx.x < a.steps * 6) steps[threadIdx.x] = (&a.step[0][0])[threadIdx.x];
  float r = a.unit.unit, trace = 0.f;
  uint32_t most = 0;
  if (r == 0.f) {   // under way beside the sums
    static_assert(kMaxSplits * kWaves <= kThreads, "a number of the trace for each thread");
    if ((int)threadIdx.x < g.splits * kWaves) trace = reinterpret_cast<const float*>(own + g.trace)[threadIdx.x];
    most = most_of(reinterpret_cast<const uint32_t*>(own + g.most), g.blocks);
  }
  // chunk c (16 bytes) of row i; columns k .. of a pair row lie in chunks of 8
  auto chunk = [&](int m, int i, int c) { return sm[m] + i * kLd + ((c ^ (i & 15)) << 4); };
  auto put = [&](int m, int i, int k, const float* v) {   // four columns
    f16x4 h, l;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f16 x, y;
      split(v[e], x, y);
      h[e] = x;
      l[e] = y;
    }
    const int c = (k >> 5) * 8 + ((k & 31) >> 3);
    *reinterpret_cast<f16x4*>(chunk(m, i, c) + (k & 4) * 2) = h;
    *reinterpret_cast<f16x4*>(chunk(m, i, c + 4) + (k & 4) * 2) = l;
  };
  auto get = [&](int m, int i, int k, float* v) {
    const int c = (k >> 5) * 8 + ((k & 31) >> 3);
    const f16x4 h = *reinterpret_cast<const f16x4*>(chunk(m, i, c) + (k & 4) * 2);
    const f16x4 l = *reinterpret_cast<const f16x4*>(chunk(m, i, c + 4) + (k & 4) * 2);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)h[e] + (float)l[e];
  };
  constexpr int S = 0, P = 1, R = 2;
  int Q = 3, other = 4;   // where Q is, and where it goes next
  const float* part = reinterpret_cast<const float*>(own + g.part);
  constexpr int kMine = kN * kN / 4 / kThreads;
  double sums[kMine][4] = {};
  for (int s = 0; s < g.splits; s += 4) {   // every load of four splits in flight
    f32x4 w[kMine][4];
#pragma unroll
    for (int u = 0; u < kMine; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[u][q] = *reinterpret_cast<const f32x4*>(part + (int64_t)min(s + q, g.splits - 1) * kN * kN +
                                                  (u * kThreads + threadIdx.x) * 4);
#pragma unroll
    for (int u = 0; u < kMine; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (s + q < g.splits)
#pragma unroll
          for (int e = 0; e < 4; ++e) sums[u][e] += (double)w[u][q][e];
  }
  if (r == 0.f) {
    float sum[1] = {trace};
    block_sum<kThreads / 64, 1>(sum, lds);
    r = norm_factor(sum[0], a.unit, most, lds_most);
  }
  if (threadIdx.x == 0 && a.scale) *reinterpret_cast<float*>(own + g.scale) = r;
#pragma unroll
  for (int u = 0; u < kMine; ++u) {
    const int x = u * kThreads + threadIdx.x;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)sums[u][e] * r * r * a.to;
    put(S, x / 16, x % 16 * 4, v);
  }
  __syncthreads();
  // The upper triangle's values on both sides: S is symmetric.  (Every read of LDS before the first
  // write, here and below: the compiler cannot tell them apart, and would wait for each in turn.)
  f16 high[kMine][4], deep[kMine][4];
#pragma unroll
  for (int u = 0; u < kMine; ++u) {
    const int x = u * kThreads + threadIdx.x, i = x / 16, j = x % 16 * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = min(j + e, i), col = max(j + e, i), c = (col >> 5) * 8 + ((col & 31) >> 3);
      high[u][e] = *reinterpret_cast<const f16*>(chunk(S, row, c) + (col & 7) * 2);
      deep[u][e] = *reinterpret_cast<const f16*>(chunk(S, row, c + 4) + (col & 7) * 2);
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kMine; ++u) {
    const int x = u * kThreads + threadIdx.x, i = x / 16, j = x % 16 * 4, c = (j >> 5) * 8 + ((j & 31) >> 3);
    *reinterpret_cast<f16x4*>(chunk(S, i, c) + (j & 4) * 2) = f16x4{high[u][0], high[u][1], high[u][2], high[u][3]};
    *reinterpret_cast<f16x4*>(chunk(S, i, c + 4) + (j & 4) * 2) = f16x4{deep[u][0], deep[u][1], deep[u][2], deep[u][3]};
  }
  const int rowa = (wave & 1) * 32 + (lane & 31), rowb = (wave >> 1) * 32 + (lane & 31);
  struct Fragments {
    f16x8 h[4], l[4];
  };
  auto fetch = [&](int m, int row, Fragments& f) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = (u >> 1) * 8 + (u & 1) * 2 + (lane >> 5);
      f.h[u] = *reinterpret_cast<const f16x8*>(chunk(m, row, c));
      f.l[u] = *reinterpret_cast<const f16x8*>(chunk(m, row, c + 4));
    }
  };
  auto product = [&](const Fragments& x, const Fragments& y, f32x16& acc) {
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
    f32x16 low = acc, also = acc;   // three sums that do not wait for each other
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      low = __builtin_amdgcn_mfma_f32_32x32x16_f16(y.h[u], x.l[u], low, 0, 0, 0);
      also = __builtin_amdgcn_mfma_f32_32x32x16_f16(y.l[u], x.h[u], also, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(y.h[u], x.h[u], acc, 0, 0, 0);
    }
    acc += low + also;
  };
  // fn(which, row, first of four columns), and also their values
  auto at_each = [&](auto fn) {
#pragma unroll
    for (int q = 0; q < 4; ++q) fn(q, (wave & 1) * 32 + (lane & 31), (wave >> 1) * 32 + 8 * q + 4 * (lane >> 5));
  };
  auto each = [&](const f32x16& acc, auto fn) {
    at_each([&](int q, int i, int j) {
      float v[4] = {acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
      fn(q, i, j, v);
    });
  };
  f32x16 x, y;
  Fragments fp, fs, f;   // P's rows, S's other rows, and what else is met
  for (int k = 0; k < a.steps; ++k) {
    const bool last = k + 1 == a.steps;
    __syncthreads();
    float of[6], s[4][4];
#pragma unroll
    for (int i = 0; i < 6; ++i) of[i] = steps[k * 6 + i];
    fetch(S, rowa, f);
    fetch(S, rowb, fs);
    at_each([&](int q, int i, int j) { get(S, i, j, s[q]); });
    product(f, fs, x);
    const int p = k == 0 ? Q : P;   // the first P is Q
    each(x, [&](int q, int i, int j, float* v) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = fmaf(of[1], s[q][e], v[e] * of[0]);
        if (i == j + e && i < n) v[e] += of[2];
      }
      put(p, i, j, v);
    });
    __syncthreads();
    fetch(p, rowa, fp);
    if (k > 0) {
      fetch(Q, rowb, f);
      product(fp, f, y);
    }
    if (!last) product(fp, fs, x);
    if (k > 0) {
      each(y, [&](int, int i, int j, float* v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= of[4];
        put(other, i, j, v);
      });
      const int was = Q;
      Q = other;
      other = was;
    }
    if (last) break;
    each(x, [&](int, int i, int j, float* v) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= of[3];
      put(R, i, j, v);
    });
    __syncthreads();
    fetch(R, rowb, f);
    product(fp, f, x);
    each(x, [&](int, int i, int j, float* v) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= of[5];
      put(S, i, j, v);
    });
  }
  __syncthreads();
  f16* out = reinterpret_cast<f16*>(square_of(g, own, a.q));
#pragma unroll
  for (int u = 0; u < kN * 16 / kThreads; ++u) {
    const int t = u * kThreads + threadIdx.x, i = t / 16, c = t % 16;
    const f16x8 v = *reinterpret_cast<const f16x8*>(chunk(Q, i, c));
    // flat: 32 columns of a block, then the lo 64 columns on
    const int at = a.form == kPair ? c * 8 : (c >> 3) * 32 + (c & 3) * 8 + ((c & 4) ? kN : 0);
    *reinterpret_cast<f16x8*>(out + i * 2 * kN + at) = v;
  }
}

// ---- Q X ----------------------------------------------------------------------------------------
// Where a matrix's result goes: `out`, or the parameter (and its master) that it updates.
struct Sink {
  void* out;
  float* master;
};
struct Sinks {
  Groups groups;
  int first;
  uint32_t total;
  Sink s[kMaxMatrices];
  float rate[kMaxMatrices];   // lr times the matrix's own factor
  int q;               // which of sq is Q
  float unit;          // 1 / Q's factor
  bool second;         // the X formed on the way
  float decay, rest;   // 1 - lr weight_decay and what its rounding leaves
};
enum Result { kOut, kParam, kMaster };

// A tile of Q X, or of X Q for a tall X, at (row0, col0) of X.
template <int T, int RING, Form F>
__device__ __forceinline__ void last_product(uint8_t* sm, const Group& g, uint8_t* own, int q,
                                             bool second, int64_t row0, int64_t col0,
                                             f32x16 (&acc)[T / 64][T / 64]) {
  // Q's rows are pairs where X's are; else all hi and then all lo against X twice
  constexpr bool PAIR = F == kPair;
  constexpr int kSize = PAIR ? 4 : 2;
  using P = Product<T, RING, F, 4, T == 64 ? 2 : 1>;
  const int64_t ld_q = (int64_t)g.nt * 4, ld_x = (int64_t)(g.tall ? g.nt : g.mt) * kSize;
  const int sq = g.ne / kPairBlock, sx = PAIR ? sq : sq / 2;
  const uint8_t* x = own + (second ? g.x2 : g.x);
  const uint8_t* qp = square_of(g, own, q);
  if (g.tall)
    P::run(sm, Side{x + row0 * ld_x, ld_x, sx}, Side{qp + col0 * ld_q, ld_q, sq}, 0, sq, acc);
  else
    P::template run<false, true>(sm, Side{qp + row0 * ld_q, ld_q, sq},
                                 Side{x + col0 * kSize, ld_x, sx}, 0, sq, acc);
}

// What the parameter was where a tile from (row0, col0) of X on will go: read before the products.
// Behind them each line would wait for its own, since the stores between cannot be told apart from the
// loads (56 layers' masters, in dora_orthogonal_last, 113 us, so 119; 24 high-rank layers' step is level).
template <typename P, bool BF, Result WHAT>
__device__ __forceinline__ void read_before(const Sinks& a, const Where& here, int64_t row0, int64_t col0,
                                            int rows, int cols, float (&before)[P::kLines][8]) {
  if (WHAT == kOut) return;
  const Sink s = a.s[here.slot];
  P::numbered([&](int n, int r, int c) {
    const int64_t i = row0 + r, j = col0 + c, at = i * cols + j, stop = (i + 1) * cols;
    if (i >= rows || j >= cols) return;
    if (WHAT == kMaster) load8<false>(s.master, at, stop, before[n]);
    else load8<BF>(s.out, at, stop, before[n]);
  });
}
// A tile of the last product in LDS to where it goes; f: its factor.
template <typename P, bool BF, Result WHAT>
__device__ __forceinline__ void put_out(float* tile, const Sinks& a, const Where& here, int64_t row0,
                                        int64_t col0, int rows, int cols, float f,
                                        const float (&before)[P::kLines][8]) {
  using E = Elem<BF>;
  const Sink s = a.s[here.slot];
  if (WHAT != kOut) f *= -a.rate[here.slot];
  typename E::T* out = reinterpret_cast<typename E::T*>(s.out);
  P::numbered([&](int n, int r, int c) {
    const int64_t i = row0 + r, j = col0 + c;
    if (i >= rows || j >= cols) return;
    float v[8];
    P::row8(tile, r, c, v);
    const int64_t at = i * cols + j, stop = (i + 1) * cols;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= f;
    if (WHAT != kOut) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = fmaf(before[n][e], a.decay, fmaf(before[n][e], a.rest, v[e]));
      if (WHAT == kMaster) {
        store_part<false>(s.master, at, stop, v);
        store_part<false>(s.master, at + 4, stop, v + 4);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; e += E::kN) store_part<BF>(out, at + e, stop, v + e);
  });
}

template <int T, int RING, Form F, bool BF, Result WHAT>
__global__ __launch_bounds__(kThreads) void dora_orthogonal_apply(const Sinks a, uint8_t* ws) {
  using P = Product<T, RING, F, 4, T == 64 ? 2 : 1>;
  __shared__ __attribute__((aligned(1024))) uint8_t sm[P::kLds];
  const uint32_t id = by_xcd(blockIdx.x, a.total);
  const Where here = where(a.groups, a.first, id, ws);
  const Group& g = here.g;
  uint8_t* own = here.own;
  const bool tall = g.tall;
  const int rows = tall ? g.m : g.n, cols = tall ? g.n : g.m;
  const int down = (rows + T - 1) / T, across = (cols + T - 1) / T;
  const int t = here.piece;
  // tiles that share X's columns next to each other
  const int64_t row0 = (int64_t)(tall ? t / across : t % down) * T;
  const int64_t col0 = (int64_t)(tall ? t % across : t / down) * T;
  float before[P::kLines][8];
  read_before<P, BF, WHAT>(a, here, row0, col0, rows, cols, before);
  const float f = *reinterpret_cast<const float*>(own + g.scale) * a.unit;
  f32x16 acc[P::kB][P::kB];
  last_product<T, RING, F>(sm, g, own, a.q, a.second, row0, col0, acc);
  float* tile = P::stage(sm, acc);
  put_out<P, BF, WHAT>(tile, a, here, row0, col0, rows, cols, f, before);
}

// The last product after QS - 1 others that were not kept (n <= 64), a block of X a workgroup.  What
// the parameter was is read before the products: 56 layers' masters take 113 us (14 bytes an element:
// 3.6 TB/s), 119 when it is read behind them.
template <int QS, bool BF, Result WHAT>
__global__ __launch_bounds__(kThreads) void dora_orthogonal_last(const Sinks a, const Turns turns,
                                                                 uint8_t* ws) {
  using P = Product<64, 4, kPair>;
  __shared__ __attribute__((aligned(1024))) uint8_t sm[kPairs], made[QS - 1][kPairs];
  const uint32_t id = by_xcd(blockIdx.x, a.total);
  const Where here = where(a.groups, a.first, id, ws);
  const Group& g = here.g;
  uint8_t* own = here.own;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), qa = wave & 1, qb = wave >> 1;
  const int64_t ld = (int64_t)(g.tall ? g.nt : g.mt) * 4;
  const float f = *reinterpret_cast<const float*>(own + g.scale) * turns.unit[0];
  auto run = [&](auto tall) {
    constexpr bool TALL = decltype(tall)::value;
    Operand<64, kPair, !TALL, kWaves> x;
    x.start(Side{own + g.x, ld, 2}, 0, qb);
    Operand<64, kPair, true, kWaves> y;
    y.start(Side{nullptr, 0, 1}, 0, qb);
    issue_block<TALL>(x, own + g.x, ld, here.piece, sm);
    const int64_t on = (int64_t)here.piece * 64, row0 = TALL ? on : 0, col0 = TALL ? 0 : on;
    const int rows = TALL ? g.m : g.n, cols = TALL ? g.n : g.m;
    float before[P::kLines][8];
    read_before<P, BF, WHAT>(a, here, row0, col0, rows, cols, before);
    Rows q[QS];
#pragma unroll
    for (int i = 0; i < QS; ++i) q[i].load(g, own, i, qa * 32);
    wait_vm<0>();
    barrier_nofence();
    keep_quarter<true>(made[0], quarter_of<false>(q[0], x, sm, qb), f, qa, qb);
    wait_lds();
    barrier_nofence();
    if (QS == 3) {
      keep_quarter<true>(made[QS - 2], quarter_of<false>(q[1], y, made[0], qb), turns.unit[1], qa, qb);
      wait_lds();
      barrier_nofence();
    }
    const f32x16 acc = quarter_of<TALL>(q[QS - 1], y, made[QS - 2], qb);
    const int lane = threadIdx.x & 63;
    float* tile = reinterpret_cast<float*>(sm);   // (X has been read)
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<f32x4*>(P::at(tile, (TALL ? qb : qa) * 32 + (lane & 31),
                                      (TALL ? qa : qb) * 32 + 8 * c + 4 * (lane >> 5))) =
          f32x4{acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]};
    __syncthreads();
    put_out<P, BF, WHAT>(tile, a, here, row0, col0, rows, cols, a.unit, before);
  };
  if (g.tall) run(std::true_type());
  else run(std::false_type());
}

// Q X as pairs, in place of X from here on.
template <int T, int RING, Form F>
__global__ __launch_bounds__(kThreads) void dora_orthogonal_between(const Groups a, uint32_t total,
                                                                    int q, float unit, bool second,
                                                                    uint8_t* ws) {
  using P = Product<T, RING, F, 4, T == 64 ? 2 : 1>;
  __shared__ __attribute__((aligned(1024))) uint8_t sm[P::kLds];
  const uint32_t id = by_xcd(blockIdx.x, total);
  const Group& g = a.g[group_of(a, id)];
  const int down = ((g.tall ? g.m : g.n) + T - 1) / T, across = ((g.tall ? g.n : g.m) + T - 1) / T;
  const int rest = (int)(id - g.from);
  const int t = rest % (down * across), u = rest / (down * across);
  uint8_t* own = ws + g.base + (int64_t)u * g.stride;
  const int64_t row0 = (int64_t)(g.tall ? t / across : t % down) * T;
  const int64_t col0 = (int64_t)(g.tall ? t % across : t / down) * T;
  f32x16 acc[P::kB][P::kB];
  last_product<T, RING, F>(sm, g, own, q, second, row0, col0, acc);
  float* tile = P::stage(sm, acc);
  const float f = *reinterpret_cast<const float*>(own + g.scale) * unit;
  f16* x = reinterpret_cast<f16*>(own + (second ? g.x : g.x2));
  const int64_t ld = 2 * (int64_t)(g.tall ? g.nt : g.mt);
  P::lines([&](int r, int c) {
    float v[8];
    P::row8(tile, r, c, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= f;
    store_pair<8>(x + (row0 + r) * ld, col0 + c, v);
  });
}

static_assert(sizeof(Sinks) <= 4000 && sizeof(Chain) <= 4000 && sizeof(Sources) <= 4000 && sizeof(Squares) <= 4000,
              "kernel arguments");

// ---- host: the iteration's numbers ------------------------------------------------------------

double largest(double l, double (*f)(double, const double*), const double* abc, double q1, double q2) {
  double m = std::max(std::fabs(f(0.0, abc)), std::fabs(f(l, abc)));
  for (double x : {q1, q2})
    if (x > 0 && x < l) m = std::max(m, std::fabs(f(x, abc)));
  return m;
}
double p_of(double x, const double* k) { return k[0] + x * (k[1] + x * k[2]); }
double r_of(double x, const double* k) { return x * p_of(x, k); }
double s_of(double x, const double* k) { return x * p_of(x, k) * p_of(x, k); }
// Real roots of u + v x + w x^2 (NaN, which no comparison takes, where there are none).
void roots(double u, double v, double w, double* x) {
  if (w == 0) {
    x[0] = x[1] = -u / v;
    return;
  }
  const double d = std::sqrt(v * v - 4 * u * w);
  x[0] = (-v + d) / (2 * w);
  x[1] = (-v - d) / (2 * w);
}

// Powers of two that keep every matrix inside half precision: its eigenvalues are polynomials of
// those of the first S, which lie in [0, 1], so their bounds are known beforehand, and no entry of a
// symmetric matrix is larger than its largest eigenvalue.
struct Numbers {
  int steps;
  double abc[kMaxSteps][3];
  int s[kMaxSteps + 1], p[kMaxSteps], r[kMaxSteps], q[kMaxSteps];   // exponents
  int x[kMaxSteps + 1];
  bool anew[kMaxSteps + 1];   // Q X is formed before step k, and S anew from it
  int times;                  // how often
  bool good;
};
int exponent(double bound) {
  // 2^14 of half precision's 2^16: roundings may pass the bound a little
  return 14 - (int)std::ceil(std::log2(std::max(bound, 0x1p-24)));
}
Numbers numbers(const double* coefficients, int steps, double most) {
  Numbers z = {};
  z.steps = steps;
  z.good = false;
  double l = 1.0, q = 1.0, grown = 0.0, gain = 1.0;
  for (int k = 0; k < steps; ++k) {
    const double* abc = z.abc[k];
    for (int i = 0; i < 3; ++i) {
      z.abc[k][i] = coefficients[3 * k + i];
      if (!std::isfinite(abc[i])) return z;
    }
    const double rise = abc[0] != 0 ? std::fabs(abc[1] / abc[0]) * gain : 0.0;
    if (k > 0 && grown + rise > most) {
      z.anew[k] = true;
      ++z.times;
      grown = 0.0;
      gain = q = 1.0;
    }
    grown += abc[0] != 0 ? std::fabs(abc[1] / abc[0]) * gain : 0.0;
    gain *= abc[0] * abc[0];
    double t[2], top;
    top = -abc[1] / (2 * abc[2]);
    const double p = largest(l, p_of, abc, top, top);
    roots(abc[0], 2 * abc[1], 3 * abc[2], t);
    const double r = largest(l, r_of, abc, t[0], t[1]);
    roots(abc[0], 3 * abc[1], 5 * abc[2], t);
    const double next = largest(l, s_of, abc, t[0], t[1]);
    q *= p;
    if (!(p < 0x1p30) || !(q < 0x1p30) || !(r < 0x1p30) || !(next < 0x1p30)) return z;
    z.s[k] = exponent(l);
    z.x[k] = exponent(std::sqrt(l));
    z.p[k] = exponent(p);
    z.r[k] = exponent(r);
    z.q[k] = exponent(q);
    l = std::max(next, 0x1p-24);
    z.s[k + 1] = exponent(l);
  }
  z.good = true;
  return z;
}

// ---- host: which matrices share launches -------------------------------------------------------
struct Item {
  int64_t rows, cols;
  Source from;
  Sink to;
  float rate;
};
struct Kind {
  Form form;      // X's
  int times;      // how often Q X is formed on the way
  // n <= 64: Q X is not kept, but formed again where it is wanted
  bool folds() const { return form == kPair && times < kMostQ; }
};
struct Pass {
  bool small;               // n <= 64 throughout
  int gram, square, apply;  // tiles
  int64_t tiles, large;     // of 64 and of 128, of an n x n product
  std::vector<int> order;   // items, group by group
  Groups groups;
  size_t bytes;
};

int64_t padded(int64_t v, int to) { return (v + to - 1) / to * to; }
int tiles(int v, int tile) { return (v + tile - 1) / tile; }

void lay_out(Group& g, const Kind& k, int gram, bool small) {
  g.ne = (int)padded(g.n, 64);
  g.nt = g.n <= 64 ? 64 : (int)padded(g.n, 128);
  g.mt = (int)padded(g.m, 128);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += padded(bytes, 256);
    return here;
  };
  g.x = take((int64_t)g.nt * g.mt * (k.form != kSingle || k.times > 1 ? 4 : 2));
  g.x2 = k.times && !(small && k.folds()) ? take((int64_t)g.nt * g.mt * 4) : 0;
  g.sq = take((int64_t)g.nt * g.nt * 4 * 5);
  g.part = take((int64_t)tri(tiles(g.n, gram)) * g.splits * gram * gram * 4);
  g.trace = take((int64_t)tiles(g.n, gram) * g.splits * kWaves * 4);
  g.most = take((int64_t)g.blocks * 4);
  g.scale = take(4);
  g.stride = at;
}

// Tiles of 128 read half of what tiles of 64 read for the same products, and are taken where they
// fill the chip: this many workgroups (2048 x 6144: 877 us in all, with tiles of 64 for S and Q X 999,
// 24 matrices of 384 x 8192 503 and 581; with tiles of 128 throughout 1031 x 517 213 instead of 174).
constexpr int64_t kEnough = 256;
constexpr int64_t kFewTiles = 384;   // of a launch of n x n products
constexpr int64_t kCus = 256;
// Workgroups of the sums over m, and the least stages of 64 of one's part.  Parts cost their partial
// sums, few of them leave CUs empty or the last ones waiting: 24 layers' step 1.57 ms, with 768
// wanted 1.60; four matrices of 384 x 8192 190 us, with parts of four stages 201; with tiles of 64
// 1031 x 517 172 us, with parts of eight 177.  For n <= 64 three lie on a CU (dora_orthogonal_fold).
constexpr int64_t kWantSums = 1024, kWantSmall = 768;
constexpr int64_t kLeastPart = 8, kLeastSmall = 4;

std::vector<Pass> passes(const std::vector<Item>& items, const Kind& kind) {
  auto small = [](const Item& i) { return std::min(i.rows, i.cols); };
  std::vector<int> order;
  order.reserve(items.size());
  for (size_t i = 0; i < items.size(); ++i)
    if (small(items[i]) > 0) order.push_back((int)i);
  std::stable_sort(order.begin(), order.end(), [&](int a, int b) {
    const Item &x = items[a], &y = items[b];
    if (small(x) != small(y)) return small(x) < small(y);
    return x.rows != y.rows ? x.rows < y.rows : x.cols < y.cols;
  });
  std::vector<Pass> out;
  for (size_t at = 0; at < order.size();) {
    const Item& one = items[order[at]];
    size_t end = at;
    while (end < order.size() && items[order[end]].rows == one.rows && items[order[end]].cols == one.cols)
      ++end;
    const bool low = small(one) <= 64;
    if (out.empty() || out.back().small != low || out.back().groups.count == kMaxGroups) {
      out.emplace_back();
      out.back().small = low;
      out.back().groups.count = 0;
    }
    Pass& p = out.back();
    Group& g = p.groups.g[p.groups.count++];
    g = Group{};
    g.n = (int)small(one);
    g.m = (int)std::max(one.rows, one.cols);
    g.tall = one.rows > one.cols;
    g.count = (int)(end - at);
    g.first = (int)p.order.size();
    p.order.insert(p.order.end(), order.begin() + at, order.begin() + end);
    at = end;
  }
  for (Pass& p : out) {
    int64_t squares = 0, across = 0, parts = 0;   // workgroups with tiles of 128
    int64_t small_squares = 0;                    // and of 64
    for (int i = 0; i < p.groups.count; ++i) {
      const Group& g = p.groups.g[i];
      const int64_t t = (int64_t)g.count * tri(tiles(g.n, 128));
      squares += t;
      small_squares += (int64_t)g.count * tri(tiles(g.n, 64));
      parts += t * std::min<int64_t>(tiles(g.m, 256), kMaxParts);
      across += (int64_t)g.count * tiles(g.n, 128) * tiles(g.m, 128);
    }
    p.gram = !p.small && parts >= kEnough ? 128 : 64;
    p.square = squares >= 2 * kEnough ? 128 : 64;
    p.tiles = small_squares;
    p.large = squares;
    p.apply = !p.small && across >= kEnough ? 128 : 64;
    int64_t stages = 0;   // of 64 of the longer side, for all tiles of S
    for (int i = 0; i < p.groups.count; ++i) {
      const Group& g = p.groups.g[i];
      stages += (int64_t)g.count * tri(tiles(g.n, p.gram)) * tiles(g.m, 64);
    }
    const int64_t want = p.small ? kWantSmall : kWantSums;
    const int64_t part = std::max<int64_t>(p.gram == 128 ? kLeastPart : kLeastSmall, (stages + want - 1) / want);
    int64_t base = 0;
    for (int i = 0; i < p.groups.count; ++i) {
      Group& g = p.groups.g[i];
      g.splits = (int)std::min<int64_t>(std::max<int64_t>(1, tiles(g.m, 64) / part),
                                        p.small ? kMaxSplits : kMaxParts);
      g.blocks = (int)std::min<int64_t>(kMaxBlocks, ((int64_t)g.n * g.m + 8191) / 8192);
      lay_out(g, kind, p.gram, p.small);
      g.base = base;
      base += g.stride * g.count;
    }
    p.bytes = (size_t)base;
  }
  return out;
}

// Sets each group's first workgroup and returns their number; size(group): of one matrix.
template <typename Size>
int64_t spread(Groups& a, Size size) {
  int64_t at = 0;
  for (int i = 0; i < a.count; ++i) {
    a.g[i].from = (uint32_t)at;
    at += size(a.g[i]) * a.g[i].count;
  }
  return at;
}

// ---- host: launches ------------------------------------------------------------------------------
struct Call {
  bool x_bf, moment, out_bf;
  Result what;
  float eps, mu, nu, decay, rest;
  int nesterov;
};

// (an argument's type is the kernel's, not what is passed)
template <typename T>
struct Identity {
  using type = T;
};
template <typename T>
using identity_t = typename Identity<T>::type;

template <int THREADS = kThreads, typename... Args>
hipError_t launch(const char* label, void (*kernel)(Args...), int64_t blocks, hipStream_t st,
                  identity_t<Args>... args) {
  LaunchTimer timer(label, st);
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(THREADS), 0, st, args...);
  return hipGetLastError();
}

// Launches over the matrices of a pass whose addresses the kernel takes; fill(slot, item).
template <typename A, typename Size, typename Fill, typename Go>
hipError_t by_matrix(const Pass& p, A& a, Size size, Fill fill, Go go) {
  a.groups = p.groups;
  const int all = (int)p.order.size();
  for (int first = 0; first < all;) {
    int64_t blocks = 0;
    int slot = 0;
    a.first = first;
    for (int i = 0; i < a.groups.count; ++i) {   // (groups of which it has none get no workgroups)
      Group& g = a.groups.g[i];
      g.from = (uint32_t)blocks;
      g.each = (int)size(g);
      g.begin = first;
      for (; first >= g.first && first < g.first + g.count && slot < kMaxMatrices; ++first) {
        if (slot && blocks + g.each > launch_blocks(kThreads)) break;
        fill(slot++, p.order[first]);
        blocks += g.each;
      }
    }
    if (hipError_t e = go(blocks)) return e;
  }
  return hipSuccess;
}

#define ORTHO_TRY(expr)                              \
  do {                                               \
    if (hipError_t e_ = (expr)) return e_;           \
  } while (0)

float two(int e) { return std::ldexp(1.f, e); }

// Stages in flight: two of a 128 tile (64 KB) leave room for a second workgroup on the CU.
constexpr int ring(int tile) { return tile == 128 ? 2 : 4; }

template <typename Fn>
hipError_t by_tile(int tile, Fn fn) {
  return tile == 128 ? fn(std::integral_constant<int, 128>()) : fn(std::integral_constant<int, 64>());
}
struct Engine {
  const Pass& p;
  const std::vector<Item>& items;
  const Numbers& z;
  const Call& c;
  Form form;     // of the current X, and which of the two it is
  bool second;
  bool folds;    // Kind's
  uint8_t* ws;
  hipStream_t st;
  // Where products are formed again (`folds`): how many there are, their factors, and the exponent
  // of what they leave.
  int seen = 0, at = 0;
  Turns turns = {};

  template <bool BF, bool MOMENT, Form F>
  hipError_t halves() {
    Sources a;
    a.mu = c.mu;
    a.nu = c.nu;
    a.nesterov = c.nesterov;
    auto fill = [&](int slot, int item) { a.s[slot] = items[item].from; };
    ORTHO_TRY(by_matrix(p, a, [](const Group& g) { return (int64_t)g.blocks; }, fill, [&](int64_t blocks) {
      return launch("orthogonal_most", dora_orthogonal_most<BF, MOMENT>, blocks, st, a, ws);
    }));
    if (p.small)
      return by_matrix(p, a, [](const Group& g) { return (int64_t)g.splits; }, fill, [&](int64_t blocks) {
        return launch("orthogonal_first", dora_orthogonal_first<BF, MOMENT, F>, blocks, st, a, ws);
      });
    return by_matrix(p, a, [](const Group& g) { return ((int64_t)g.nt * g.mt + kPiece - 1) / kPiece; }, fill,
                     [&](int64_t blocks) {
                       return launch("orthogonal_halves", dora_orthogonal_halves<BF, MOMENT, F>, blocks, st, a, ws);
                     });
  }
  hipError_t start() {
    if (c.moment) return c.x_bf ? halves<true, true, kPair>() : halves<false, true, kPair>();
    return c.x_bf ? halves<true, false, kSingle>() : halves<false, false, kPair>();
  }
  Unit unit_of(float unit) const { return {unit, c.eps}; }
  // fn with X's form, one of FORMS, as a constant
  template <Form... FORMS, typename Fn>
  hipError_t by_form(Fn fn) const {
    hipError_t e = hipErrorInvalidValue;
    (void)((form == FORMS && (e = fn(std::integral_constant<Form, FORMS>()), true)) || ...);
    return e;
  }

  // S of the current X; `unit` as dora_orthogonal_gather takes it
  hipError_t gram(float unit, int to) {
    return by_tile(p.gram, [&](auto tile) {
      constexpr int T = decltype(tile)::value;
      Groups a = p.groups;
      int64_t blocks = spread(a, [](const Group& g) { return (int64_t)tri(tiles(g.n, T)) * g.splits; });
      ORTHO_TRY((by_form<kSingle, kPair>([&](auto f) {
        return launch("orthogonal_gram", dora_orthogonal_gram<T, ring(T), decltype(f)::value>, blocks,
                      st, a, (uint32_t)blocks, second, ws);
      })));
      if (p.small) return hipSuccess;   // the chain gathers it
      blocks = spread(a, [](const Group& g) {
        return (int64_t)tri(tiles(g.n, T)) * (T / 32) * (T / 32);
      });
      return launch("orthogonal_gather", dora_orthogonal_gather<T>, blocks, st, a,
                    unit_of(unit), two(to), ws);
    });
  }
  template <bool POLY, int T, int RING, int WAVES, int DEEP>
  hipError_t squares_on(const Square& one, const Square* two) {
    Squares a;
    a.groups = p.groups;
    const int64_t blocks = spread(a.groups, [](const Group& g) { return (int64_t)tri(tiles(g.n, T)); });
    a.half = (uint32_t)blocks;
    a.total = (uint32_t)(two ? 2 * blocks : blocks);
    a.q[0] = one;
    a.q[1] = two ? *two : one;
    return launch<WAVES * 64>(POLY ? "orthogonal_poly" : "orthogonal_square",
                              dora_orthogonal_square<T, RING, WAVES, DEEP, POLY>, a.total, st, a, ws);
  }
  // Tiles of 64 in two stages (32 KB) lie five to a CU: 48 matrices of 384 take 24 us a product, with
  // tiles of 128 30; a matrix of 2048 takes 48 and 58.  From two of the large tiles for each CU on
  // their half traffic counts (4096 columns: 4.6 ms in all against 5.0, 5000: 7.9 against 10.2).  Fewer
  // of them are worth it where they leave the fullest CU no more work than tiles of 64 do, one to a CU
  // in four stages (1800 columns: 604 us against 631, 2600: 1342 against 1427; 2048, where they do not,
  // 990 against 905; 40 matrices of 384, where it is level: 518 against 515).  Few tiles have the CU's
  // SIMDs to themselves: eight waves, and two stages at a time, since a stage is 750 cycles of waiting
  // for LDS and for each other (517 columns: 175 us in all, one stage at a time 184, four waves 192; 1536
  // columns, whose double launches have 600 tiles: 467 us either way; 24 matrices of 384, 504 tiles: 335
  // us as here, 355 with eight waves).
  template <bool POLY>
  hipError_t squares(const Square& one, const Square* two = nullptr) {
    if (p.square == 128) return squares_on<POLY, 128, 2, 8, 1>(one, two);
    const int64_t small = p.tiles * (two ? 2 : 1), large = p.large * (two ? 2 : 1);
    if (small <= kFewTiles) return squares_on<POLY, 64, 4, 8, 2>(one, two);
    const int64_t each = (small + kCus - 1) / kCus, each_large = (large + kCus - 1) / kCus;
    return 4 * each_large <= each ? squares_on<POLY, 128, 4, 8, 1>(one, two)
                                  : squares_on<POLY, 64, 2, 4, 1>(one, two);
  }
  hipError_t fold() {
    Groups a = p.groups;
    const int64_t blocks = spread(a, [](const Group& g) { return (int64_t)g.splits; });
    return launch("orthogonal_fold", seen == 1 ? dora_orthogonal_fold<1> : dora_orthogonal_fold<2>, blocks, st, a,
                  (uint32_t)blocks, turns, ws);
  }
  hipError_t between(int q, int e) {
    ORTHO_TRY(by_tile(p.apply, [&](auto tile) {
      constexpr int T = decltype(tile)::value;
      Groups a = p.groups;
      const int64_t blocks =
          spread(a, [](const Group& g) { return (int64_t)tiles(g.n, T) * tiles(g.m, T); });
      return by_form<kSingle, kPair>([&](auto f) {
        return launch("orthogonal_between", dora_orthogonal_between<T, ring(T), decltype(f)::value>,
                      blocks, st, a, (uint32_t)blocks, q, two(e), second, ws);
      });
    }));
    form = kPair;
    second = !second;
    return hipSuccess;
  }
  template <bool BF, Result WHAT, Form... FORMS>
  hipError_t apply(int q, int e) {
    Sinks a;
    a.q = q;
    a.unit = two(-e - at);
    a.second = second;
    a.decay = c.decay;
    a.rest = c.rest;
    auto fill = [&](int slot, int item) {
      a.s[slot] = items[item].to;
      a.rate[slot] = items[item].rate;
    };
    if constexpr (!BF || WHAT != kOut)   // (bf16 matrices keep what they form)
      if (seen > 0)
        return by_matrix(p, a, [](const Group& g) { return (int64_t)tiles(g.m, 64); }, fill, [&](int64_t blocks) {
          a.total = (uint32_t)blocks;
          return launch("orthogonal_apply",
                        seen == 1 ? dora_orthogonal_last<2, BF, WHAT> : dora_orthogonal_last<3, BF, WHAT>,
                        blocks, st, a, turns, ws);
        });
    return by_tile(p.apply, [&](auto tile) {
      return by_form<FORMS...>([&](auto f) {
        constexpr int T = decltype(tile)::value;
        auto size = [](const Group& g) { return (int64_t)tiles(g.n, T) * tiles(g.m, T); };
        return by_matrix(p, a, size, fill, [&](int64_t blocks) {
          a.total = (uint32_t)blocks;
          return launch("orthogonal_apply",
                        dora_orthogonal_apply<T, ring(T), decltype(f)::value, BF, WHAT>, blocks,
                        st, a, ws);
        });
      });
    });
  }
  // (kPair where X was formed on the way)
  hipError_t finish(int q, int e) {
    if (c.what == kMaster) return apply<true, kMaster, kPair>(q, e);
    if (c.what == kParam)
      return c.out_bf ? apply<true, kParam, kPair>(q, e) : apply<false, kParam, kPair>(q, e);
    return c.out_bf ? apply<true, kOut, kSingle, kPair>(q, e) : apply<false, kOut, kPair>(q, e);
  }

  // The steps [from, to) between two products with X, from S's partial sums; which of sq is Q and
  // its exponent in q and e.
  hipError_t chain(int from, int to, float unit, int& q, int& e) {
    Chain a;
    a.groups = p.groups;
    a.steps = to - from;
    a.unit = unit_of(unit);
    a.to = two(z.s[from]);
    a.form = form;
    a.q = seen;
    a.scale = seen == 0;
    e = z.p[from];
    for (int k = from; k < to; ++k) {
      const int i = k - from;
      float* of = a.step[i];
      of[0] = (float)std::ldexp(z.abc[k][2], z.p[k] - 2 * z.s[k]);
      of[1] = (float)std::ldexp(z.abc[k][1], z.p[k] - z.s[k]);
      of[2] = (float)std::ldexp(z.abc[k][0], z.p[k]);
      of[3] = two(z.r[k] - z.p[k] - z.s[k]);
      of[5] = two(z.s[k + 1] - z.p[k] - z.r[k]);
      of[4] = two(z.q[k] - z.p[k] - e);
      if (i > 0) e = z.q[k];
    }
    q = 0;
    const int64_t blocks = spread(a.groups, [](const Group&) { return (int64_t)1; });
    return launch("orthogonal_chain", dora_orthogonal_chain, blocks, st, a, ws);
  }
  hipError_t products(int from, int to, int& q, int& e) {
    constexpr int S = 0, P = 1, R = 2, Qa = 3, Qb = 4;
    for (int k = from; k < to; ++k) {
      const bool last = k + 1 == to;   // Q meets X next
      const int as = last ? form : kPair;
      const int pi = k == from ? Qa : P;   // the first P is Q
      const double* abc = z.abc[k];
      Square poly = {S, S, pi, (float)std::ldexp(abc[2], z.p[k] - 2 * z.s[k]),
                     (float)std::ldexp(abc[1], z.p[k] - z.s[k]), (float)std::ldexp(abc[0], z.p[k]),
                     k == from ? as : kPair};
      ORTHO_TRY(squares<true>(poly));
      const Square ps = {pi, S, R, two(z.r[k] - z.p[k] - z.s[k]), 0.f, 0.f, kPair};
      if (k == from) {
        q = Qa;
        e = z.p[k];
        if (!last) ORTHO_TRY(squares<false>(ps));
      } else {
        const int next = q == Qa ? Qb : Qa;
        const Square pq = {P, q, next, two(z.q[k] - z.p[k] - e), 0.f, 0.f, as};
        ORTHO_TRY(squares<false>(pq, last ? nullptr : &ps));
        q = next;
        e = z.q[k];
      }
      if (!last)
        ORTHO_TRY(squares<false>(Square{pi, R, S, two(z.s[k + 1] - z.p[k] - z.r[k]), 0.f, 0.f, kPair}));
    }
    return hipSuccess;
  }

  hipError_t run() {
    ORTHO_TRY(start());
    for (int from = 0; from < z.steps;) {
      int to = from + 1;
      while (to < z.steps && !z.anew[to]) ++to;
      const float unit = from ? two(-z.x[from]) : 0.f;
      // (for n <= 64 the pass that writes X, or takes it on, has formed S)
      if (!p.small || (from && !folds)) ORTHO_TRY(gram(unit, z.s[from]));
      int q = 0, e = 0;
      ORTHO_TRY(p.small ? chain(from, to, unit, q, e) : products(from, to, q, e));
      if (to == z.steps) return finish(q, e);
      if (folds) {
        turns.unit[seen++] = two(z.x[to] - e - at);
        at = z.x[to];
        ORTHO_TRY(fold());
      } else {
        ORTHO_TRY(between(q, z.x[to] - e));
      }
      from = to;
    }
    return hipSuccess;
  }
};

hipError_t run_all(const std::vector<Item>& items, const Kind& kind, const Numbers& z, const Call& c,
                   void* ws, hipStream_t st) {
  for (const Pass& p : passes(items, kind)) {
    Engine e{p, items, z, c, kind.form, false, p.small && kind.folds(), reinterpret_cast<uint8_t*>(ws), st};
    ORTHO_TRY(e.run());
  }
  return hipSuccess;
}

size_t bytes_of(const std::vector<Item>& items, const Kind& kind) {
  size_t most = 0;
  for (const Pass& p : passes(items, kind)) most = std::max(most, p.bytes);
  return most;
}

// ---- host: arguments -----------------------------------------------------------------------------
bool dtype_ok(int dt) { return dt == DORA_F32 || dt == DORA_BF16; }
size_t esize(int dt) { return dt == DORA_BF16 ? 2 : 4; }

constexpr int64_t kMaxLong = int64_t(1) << 20, kMaxShort = 16384;
constexpr int64_t kMaxCount = int64_t(1) << 20;

bool sides_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 0 && std::max(rows, cols) <= kMaxLong &&
         std::min(rows, cols) <= kMaxShort;
}

int check_iteration(const dora_newton_schulz* o, double most, Numbers& z) {
  if (!(o->eps >= 0x1p-100) || !std::isfinite(o->eps) || !std::isfinite((float)o->eps) || o->steps < 1 ||
      o->steps > kMaxSteps)
    return DORA_ERR_FLAGS;
  if (!o->coefficients) return DORA_ERR_NULL;
  z = numbers(o->coefficients, o->steps, most);
  return z.good ? DORA_OK : DORA_ERR_FLAGS;
}

// The factor on S's rounding up to which Q is kept, by what the result is: float32 matrices (S anew
// after two of five usual steps, and after four), updates of float32 parameters, of which they are a
// few percent (after three: each time costs a fifth of the step of 56 rank-64 layers), and bf16
// (never in five steps).
constexpr double kMostExact = 20.0, kMostUpdate = 1024.0, kMostBrief = 65536.0;
struct Setup {
  Numbers z;
  Kind kind;
  std::vector<Item> items;
};

int set_up(const dora_orthogonalize_options* o, const dora_matrix* a, int64_t count, Setup& s) {
  if (!o) return DORA_ERR_NULL;
  if (!dtype_ok(o->dtype)) return DORA_ERR_DTYPE;
  if (o->reserved != 0) return DORA_ERR_FLAGS;
  const bool exact = o->dtype == DORA_F32;
  DORA_CHECK(check_iteration(&o->iteration, exact ? kMostExact : kMostBrief, s.z));
  if (count < 0 || count >= kMaxCount) return DORA_ERR_SHAPE;
  if (count > 0 && !a) return DORA_ERR_NULL;
  s.kind = {exact ? kPair : kSingle, s.z.times};
  s.items.resize((size_t)count);
  for (int64_t i = 0; i < count; ++i) {
    if (!sides_ok(a[i].rows, a[i].cols)) return DORA_ERR_SHAPE;
    s.items[i] = {a[i].rows, a[i].cols, {a[i].x, nullptr}, {a[i].out, nullptr}, 0.f};
  }
  return DORA_OK;
}

int set_up(const dora_muon_options* o, const dora_muon_tensor* a, int64_t count, Setup& s, bool& master) {
  if (!o) return DORA_ERR_NULL;
  if (!dtype_ok(o->param_dtype) || !dtype_ok(o->grad_dtype)) return DORA_ERR_DTYPE;
  if (o->reserved != 0 || (o->nesterov != 0 && o->nesterov != 1) || !std::isfinite(o->lr) ||
      !std::isfinite(o->weight_decay) || !(o->momentum >= 0 && o->momentum < 1))
    return DORA_ERR_FLAGS;
  if (count < 0 || count >= kMaxCount) return DORA_ERR_SHAPE;
  if (count > 0 && !a) return DORA_ERR_NULL;
  bool any = false;
  master = false;
  s.items.resize((size_t)count);
  for (int64_t i = 0; i < count; ++i) {
    if (!sides_ok(a[i].rows, a[i].cols)) return DORA_ERR_SHAPE;
    if (!std::isfinite(a[i].scale)) return DORA_ERR_FLAGS;
    s.items[i] = {a[i].rows, a[i].cols, {a[i].grad, a[i].momentum},
                  {a[i].param, a[i].master}, (float)(o->lr * a[i].scale)};
    if (a[i].rows == 0 || a[i].cols == 0) continue;
    if (!any) master = a[i].master != nullptr;
    any = true;
    if ((a[i].master != nullptr) != master) return DORA_ERR_NULL;
  }
  if (master && o->param_dtype != DORA_BF16) return DORA_ERR_DTYPE;
  const bool exact = master || o->param_dtype == DORA_F32;
  DORA_CHECK(check_iteration(&o->iteration, exact ? kMostUpdate : kMostBrief, s.z));
  s.kind = {kPair, s.z.times};
  return DORA_OK;
}

}  // namespace
}  // namespace dora

using namespace dora;

extern "C" {

DORA_API size_t dora_orthogonalize_workspace_bytes(const dora_matrix* matrices, int64_t count,
                                                   const dora_orthogonalize_options* options) {
  try {
    Setup s;
    return set_up(options, matrices, count, s) == DORA_OK ? bytes_of(s.items, s.kind) : 0;
  } catch (...) {   // no memory on the host
    return 0;
  }
}

DORA_API int dora_orthogonalize(const dora_matrix* matrices, int64_t count,
                                const dora_orthogonalize_options* options, void* ws, size_t ws_bytes,
                                void* hip_stream) {
  try {
    Setup s;
    DORA_CHECK(set_up(options, matrices, count, s));
    const size_t e = esize(options->dtype);
    for (int64_t i = 0; i < count; ++i) {
      const bool none = matrices[i].rows == 0 || matrices[i].cols == 0;
      DORA_CHECK(check_elem(matrices[i].x, e, none));
      DORA_CHECK(check_elem(matrices[i].out, e, none));
    }
    DORA_CHECK(check_ws(ws, ws_bytes, bytes_of(s.items, s.kind)));
    Call c = {};
    c.x_bf = c.out_bf = options->dtype == DORA_BF16;
    c.what = kOut;
    c.eps = (float)options->iteration.eps;
    HIP_TRY(run_all(s.items, s.kind, s.z, c, ws, reinterpret_cast<hipStream_t>(hip_stream)));
    return DORA_OK;
  } catch (...) {
    return DORA_ERR_HIP;
  }
}

DORA_API size_t dora_muon_workspace_bytes(const dora_muon_tensor* tensors, int64_t count,
                                          const dora_muon_options* options) {
  try {
    Setup s;
    bool master;
    return set_up(options, tensors, count, s, master) == DORA_OK ? bytes_of(s.items, s.kind) : 0;
  } catch (...) {
    return 0;
  }
}

DORA_API int dora_muon_step(const dora_muon_tensor* tensors, int64_t count,
                            const dora_muon_options* options, void* ws, size_t ws_bytes,
                            void* hip_stream) {
  try {
    Setup s;
    bool master;
    DORA_CHECK(set_up(options, tensors, count, s, master));
    const dora_muon_options& o = *options;
    for (int64_t i = 0; i < count; ++i) {
      const dora_muon_tensor& t = tensors[i];
      const bool none = t.rows == 0 || t.cols == 0;
      DORA_CHECK(check_elem(t.param, esize(o.param_dtype), none));
      DORA_CHECK(check_elem(t.grad, esize(o.grad_dtype), none));
      DORA_CHECK(check_elem(t.momentum, 4, none));
      DORA_CHECK(check_elem(t.master, 4, true));
    }
    DORA_CHECK(check_ws(ws, ws_bytes, bytes_of(s.items, s.kind)));
    Call c = {};
    c.x_bf = o.grad_dtype == DORA_BF16;
    c.out_bf = o.param_dtype == DORA_BF16;
    c.moment = true;
    c.what = master ? kMaster : kParam;
    c.eps = (float)o.iteration.eps;
    c.mu = (float)o.momentum;
    c.nu = (float)(1.0 - o.momentum);
    c.nesterov = o.nesterov;
    // what float32 loses of 1 - lr weight_decay beside 1 is added apart
    const double decay = o.lr * o.weight_decay;
    c.decay = (float)(1.0 - decay);
    c.rest = (float)(1.0 - decay - (double)c.decay);
    HIP_TRY(run_all(s.items, s.kind, s.z, c, ws, reinterpret_cast<hipStream_t>(hip_stream)));
    return DORA_OK;
  } catch (...) {
    return DORA_ERR_HIP;
  }
}

}  // extern "C"
