// Rows of any length and alignment: loads and stores of 16-byte vectors that
// start at any element (global memory takes unaligned 16-byte accesses on
// gfx950; a row that starts inside a cache line costs one more line per wave),
// and reductions over a wave and a workgroup.
#pragma once
#include "common.h"

namespace dora {

template <bool BF>
struct Elem;   // element type of a tensor: bf16 (8 per vector) or float32 (4)

template <>
struct Elem<true> {
  using T = uint16_t;
  static constexpr int kN = 8;
  using Vec = u32x4;
  using Word = uint32_t;   // 32 bits of a vector; its element q
  __device__ static float from_word(Word w, int q) { return (q & 1) ? bf_hi(w) : bf_lo(w); }
  typedef Vec Raw __attribute__((aligned(2)));
  __device__ static float get(const T* p) { return bf16_to_f32(*p); }
  __device__ static void put(T* p, float v) { *p = f32_to_bf16(v); }
  __device__ static Vec raw(const T* p) { return *reinterpret_cast<const Raw*>(p); }
  __device__ static Vec raw_past(const T* p) {   // past the caches
    return __builtin_nontemporal_load(reinterpret_cast<const Raw*>(p));
  }
  __device__ static Vec masked() {   // every element -inf
    return Vec{0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u};
  }
  __device__ static void decode(const Vec& v, float* out) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      out[2 * d] = bf_lo(v[d]);
      out[2 * d + 1] = bf_hi(v[d]);
    }
  }
  __device__ static void load(const T* p, float* out) { decode(raw(p), out); }
  __device__ static Vec encode(const float* in) {
    Vec v;
#pragma unroll
    for (int d = 0; d < 4; ++d) v[d] = pack_bf16x2(in[2 * d], in[2 * d + 1]);
    return v;
  }
  __device__ static void store_raw(T* p, Vec v) { *reinterpret_cast<Raw*>(p) = v; }
  __device__ static void store(T* p, const float* in) { store_raw(p, encode(in)); }
  // past the caches, for what is too large to stay in them
  __device__ static void store_through(T* p, const float* in) {
    __builtin_nontemporal_store(encode(in), reinterpret_cast<Raw*>(p));
  }
};

template <>
struct Elem<false> {
  using T = float;
  static constexpr int kN = 4;
  using Vec = f32x4;
  using Word = float;
  __device__ static float from_word(Word w, int) { return w; }
  typedef Vec Raw __attribute__((aligned(4)));
  __device__ static float get(const T* p) { return *p; }
  __device__ static void put(T* p, float v) { *p = v; }
  __device__ static Vec raw(const T* p) { return *reinterpret_cast<const Raw*>(p); }
  __device__ static Vec raw_past(const T* p) {   // past the caches
    return __builtin_nontemporal_load(reinterpret_cast<const Raw*>(p));
  }
  __device__ static Vec masked() {
    const float inf = __builtin_huge_valf();
    return Vec{-inf, -inf, -inf, -inf};
  }
  __device__ static void decode(const Vec& v, float* out) {
#pragma unroll
    for (int d = 0; d < 4; ++d) out[d] = v[d];
  }
  __device__ static void load(const T* p, float* out) { decode(raw(p), out); }
  __device__ static Vec encode(const float* in) { return Vec{in[0], in[1], in[2], in[3]}; }
  __device__ static void store_raw(T* p, Vec v) { *reinterpret_cast<Raw*>(p) = v; }
  __device__ static void store(T* p, const float* in) { store_raw(p, encode(in)); }
  // past the caches, for what is too large to stay in them
  __device__ static void store_through(T* p, const float* in) {
    __builtin_nontemporal_store(encode(in), reinterpret_cast<Raw*>(p));
  }
};

// Elements [j, j + kN) of a row of n, absent ones as `fill`.
template <bool BF>
__device__ __forceinline__ void load_part(const typename Elem<BF>::T* row, int64_t j, int64_t n,
                                          float fill, float* out) {
  using E = Elem<BF>;
  if (j + E::kN <= n) {
    E::load(row + j, out);
  } else {
#pragma unroll
    for (int q = 0; q < E::kN; ++q) out[q] = j + q < n ? E::get(row + j + q) : fill;
  }
}

template <bool BF>
__device__ __forceinline__ void store_part(typename Elem<BF>::T* row, int64_t j, int64_t n,
                                           const float* in) {
  using E = Elem<BF>;
  if (j + E::kN <= n) {
    E::store(row + j, in);
  } else {
#pragma unroll
    for (int q = 0; q < E::kN; ++q)
      if (j + q < n) E::put(row + j + q, in[q]);
  }
}

// Sum over a wave to every lane, in a fixed order: neighbours inside rows of 16
// lanes through DPP, then the four rows.  (Shuffles through LDS take several
// times as long, and the row reductions stand between a row's load and its
// store.)
template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_move<0xB1>(v);    // quad_perm 1,0,3,2
  v += dpp_move<0x4E>(v);    // quad_perm 2,3,0,1
  v += dpp_move<0x141>(v);   // row_half_mirror: the other quad of eight lanes
  v += dpp_move<0x140>(v);   // row_mirror: the other half of sixteen
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// Sums of N values over WAVES waves, in a fixed order, to every thread of them;
// `t` is the thread's number among them.  `lds` holds WAVES * N floats; a barrier
// of the whole workgroup stands between two uses of it.
template <int WAVES, int N>
__device__ __forceinline__ void group_sum(float* v, float* lds, int t) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (WAVES == 1) return;
  if ((t & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) lds[(t >> 6) * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = lds[i];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += lds[w * N + i];
    v[i] = s;
  }
}
// The same over a whole workgroup.
template <int WAVES, int N>
__device__ __forceinline__ void block_sum(float* v, float* lds) {
  group_sum<WAVES, N>(v, lds, threadIdx.x);
}

}  // namespace dora
