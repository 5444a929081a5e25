// Tokens of packed or padded sequences, walked in rounds of 256 tokens, four to a
// lane.  A round that lies in one sequence (nearly all do) costs no more than a
// flat pass; at a border the round is taken apart, one sequence after the other.
#pragma once
#include "../../include/dora_posttrain.h"
#include "elem.h"

#include <algorithm>

namespace dora {

constexpr int kRound = 256;   // tokens of a wave's round

// dora_token_batch on the device.
struct Batch {
  int64_t tokens, sequences, length;
  const int64_t* offsets;
  const uint8_t* mask;

  // The first token of sequence s, or the end of the last one for s = sequences;
  // inside [0, tokens] whatever the offsets hold.
  __device__ __forceinline__ int64_t start(int64_t s) const {
    if (!offsets) return s * length;
    const int64_t o = offsets[s];
    return o < 0 ? 0 : o > tokens ? tokens : o;
  }
  // The sequence of token t: the last one that starts at t or before, -1 before the
  // first.  `sequences` behind the last.  A whole wave looks for one t: 64 starts at a
  // time, so that 4096 sequences are two loads one after the other (of a wave's 5 us
  // on 256 tokens a search by halves of 512 took more than half).
  __device__ __forceinline__ int64_t sequence_of(int64_t t) const {
    if (!offsets) return length > 0 ? t / length : sequences;
    int64_t lo = -1, hi = sequences + 1;   // start(lo) <= t < start(hi)
    while (hi - lo > 1) {
      const int64_t step = (hi - lo + 63) / 64;
      const int64_t at = lo + (int64_t)((threadIdx.x & 63) + 1) * step;
      // lanes at hi or behind it count as behind t
      const int n = __popcll(__ballot(at < hi && start(at) <= t));
      lo += n * step;
      hi = min(hi, lo + step);
    }
    return lo;
  }
  __device__ __forceinline__ bool inside(int64_t s) const { return s >= 0 && s < sequences; }
  // Where the tokens of `s` end, for any value of sequence_of.
  __device__ __forceinline__ int64_t end(int64_t s) const {
    return s >= sequences ? tokens : start(s + 1);
  }
  // The sequence after s, for a token t that is behind s: usually the next one.
  __device__ __forceinline__ int64_t next(int64_t s, int64_t t) const {
    ++s;
    return end(s) > t ? s : sequence_of(t);
  }
};

// Which of the four tokens from t on count, as far as mask and the batch's end go.
__device__ __forceinline__ void counted(const Batch& b, int64_t t, bool* live) {
  if (t + 4 <= b.tokens) {
    uint32_t m = 0x01010101u;
    if (b.mask) __builtin_memcpy(&m, b.mask + t, 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) live[q] = (m >> (8 * q)) & 0xffu;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) live[q] = t + q < b.tokens && (!b.mask || b.mask[t + q]);
  }
}

__device__ __forceinline__ void load4(const float* p, int64_t t, int64_t n, float* v) {
  load_part<false>(p, t, n, 0.f, v);
}

// Sum over a wave to every lane, in a fixed order, as wave_sum for float32.
template <int CTRL>
__device__ __forceinline__ double dpp_move64(double v) {
  return __hiloint2double(__builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, 0xf, 0xf, true),
                          __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ double lane_value64(double v, int lane) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                          __builtin_amdgcn_readlane(__double2loint(v), lane));
}
// Sums over rows of 16 lanes, to each of their lanes.
__device__ __forceinline__ double row_sum64(double v) {
  v += dpp_move64<0xB1>(v);    // quad_perm 1,0,3,2
  v += dpp_move64<0x4E>(v);    // quad_perm 2,3,0,1
  v += dpp_move64<0x141>(v);   // row_half_mirror: the other quad of eight lanes
  return v + dpp_move64<0x140>(v);   // row_mirror: the other half of sixteen
}
__device__ __forceinline__ double wave_sum64(double v) {
  v = row_sum64(v);
  return (lane_value64(v, 0) + lane_value64(v, 16)) + (lane_value64(v, 32) + lane_value64(v, 48));
}

// Two sums over (part of) a sequence.
struct Pair64 {
  double v, n;
};

// Where the sums of sequences lie until they are joined, by chunks of tokens that
// one wave walks: a sequence that lies in one chunk has `own`; of another one the
// chunk that it begins in has the `tail`, every later one the `head`.
struct Parts {
  Pair64 *head, *tail, *own;
};

// Sums of sequence s from its parts, by a whole wave, in a fixed order.
__device__ __forceinline__ Pair64 join(const Batch& b, const Parts& p, int64_t s, int64_t chunk) {
  const int64_t from = b.start(s), to = b.end(s);
  if (from >= to) return {0.0, 0.0};
  const int64_t c0 = from / chunk, c1 = (to - 1) / chunk;
  if (c0 == c1) return p.own[s];
  Pair64 sum = {0.0, 0.0};
  for (int64_t c = c0 + (threadIdx.x & 63); c <= c1; c += 64) {
    const Pair64 x = c == c0 ? p.tail[c] : p.head[c];
    sum.v += x.v;
    sum.n += x.n;
  }
  return {wave_sum64(sum.v), wave_sum64(sum.n)};
}

// The sequence that a wave has come to, where it ends, and whether it began in the
// wave's chunk.
struct Cursor {
  int64_t s, end;
  bool began;
};
__device__ __forceinline__ Cursor cursor_at(const Batch& b, int64_t c0) {
  Cursor c;
  c.s = b.sequence_of(c0);
  c.end = b.end(c.s);
  c.began = b.inside(c.s) && b.start(c.s) >= c0;
  return c;
}

// Takes the cursor through the tokens [r0, r1) of a round in a chunk that ends at c1:
//   part(s, from, to)   tokens [from, to) of them are sequence s's (a real one)
//   ended(s, began)     it has no more tokens
// Each step raises s, so that it ends whatever the offsets hold.
template <typename Part, typename Ended>
__device__ __forceinline__ void through_round(const Batch& b, Cursor& c, int64_t r0, int64_t r1,
                                              int64_t c1, Part part, Ended ended) {
  int64_t pos = r0;
  while (true) {
    if (b.inside(c.s)) part(c.s, pos, min(c.end, r1));
    if (c.end > r1 || c.s >= b.sequences) return;
    if (b.inside(c.s)) ended(c.s, c.began);
    pos = max(pos, c.end);
    c.s = c.end >= c1 ? b.sequences : max(b.next(c.s, pos), c.s + 1);
    c.end = b.end(c.s);
    c.began = true;
  }
}

// ---- host ---------------------------------------------------------------------------
constexpr int64_t kMaxTokens = int64_t(1) << 34;
constexpr int64_t kMaxSequences = int64_t(1) << 31;

inline int check_batch(const dora_token_batch* b) {
  if (!b) return DORA_ERR_NULL;
  if (b->tokens < 0 || b->tokens >= kMaxTokens || b->sequences < 0 ||
      b->sequences >= kMaxSequences || b->length < 0)
    return DORA_ERR_SHAPE;
  if (b->offsets ? b->length != 0
                 : (b->sequences > 0 ? b->tokens % b->sequences != 0 ||
                                           b->tokens / b->sequences != b->length
                                     : b->tokens != 0))
    return DORA_ERR_SHAPE;
  return reinterpret_cast<uintptr_t>(b->offsets) % 8 ? DORA_ERR_ALIGN : DORA_OK;
}

inline Batch device_batch(const dora_token_batch& b) {
  return {b.tokens, b.sequences, b.length, b.offsets, b.mask};
}

// Tokens of a wave's chunk: one round until there are `most` of them.  Sums leave parts of each
// chunk behind; the policy's gradient leaves nothing, and waves of one round hide each other's loads best (4.2M
// tokens' policy gradient, over and over on the same tokens, 20.0 us, with four rounds a wave 21.2).
constexpr int64_t kMostSums = 4096, kMostGrads = int64_t(1) << 22;
inline int64_t chunk_of(int64_t tokens, int64_t most) {
  const int64_t rounds = (tokens + kRound - 1) / kRound;
  return std::max<int64_t>(1, (rounds + most - 1) / most) * kRound;
}
inline int64_t chunks_of(int64_t tokens, int64_t most) {
  const int64_t c = chunk_of(tokens, most);
  return (tokens + c - 1) / c;
}

}  // namespace dora
