// How the many tensors of a call are cut into launches, on the host.  HIP holds
// the threads of a launch below 2^32.
#pragma once
#include <stdint.h>

#include <algorithm>

namespace dora {

// The most workgroups of so many threads in one launch.
constexpr int64_t launch_blocks(int threads) { return (int64_t(1) << 31) / threads; }

// Cuts tensors of size(i) elements, i in [0, count), into pieces of whole chunks, and
// the pieces into launches of at most `tensors` pieces and `most` workgroups, one to
// a chunk:
//   add(slot, i, at, n, block)  elements [at, at + n) of tensor i are piece `slot` of
//                               the next launch, from its workgroup `block` on
//   launch(pieces, blocks)      launches them; an error (not 0) ends the cutting
// A tensor that fits one launch is one piece.  Empty tensors are left out.
template <typename Error, typename Size, typename Add, typename Launch>
Error cut_launches(int64_t count, int64_t chunk, int tensors, int64_t most, Size size, Add add,
                   Launch launch) {
  int slot = 0;
  int64_t blocks = 0;
  for (int64_t i = 0; i < count; ++i) {
    const int64_t all = size(i);
    for (int64_t at = 0; at < all;) {
      const int64_t n = std::min(all - at, most * chunk);
      const int64_t c = (n + chunk - 1) / chunk;
      if (slot == tensors || blocks + c > most) {
        if (Error e = launch(slot, blocks)) return e;
        slot = 0;
        blocks = 0;
      }
      add(slot++, i, at, n, blocks);
      blocks += c;
      at += n;
    }
  }
  return slot ? launch(slot, blocks) : Error();
}

}  // namespace dora
