// Host-side planning of the norm and the 4-bit products: pure C++ with no HIP dependency, so that
// it can be built and checked on its own.
#pragma once
#include "sffn_i8_host.h"

namespace sffn {
namespace host {

// Activations in 4-bit blocks in scratch: rows of whole groups of 16 blocks (512 values: 256 bytes
// of codes, 16 of scales), the blocks past a row's end zeros.
constexpr int kMx4Group = 16;
inline int mx4_blocks(int K) { return (int)(((int64_t)K + 31) / 32); }
inline int mx4_padded(int K) { return (int)up_to((size_t)mx4_blocks(K), kMx4Group); }

struct Mx4Carve {
  size_t q, scale, bytes;
};
inline Mx4Carve mx4_carve(size_t M, int K) {
  Mx4Carve c{};
  c.q = 0;
  c.scale = up_to(M * (size_t)mx4_padded(K) * 16, 256);
  c.bytes = c.scale + up_to(M * (size_t)mx4_padded(K), 256);
  return c;
}

}  // namespace host
}  // namespace sffn
