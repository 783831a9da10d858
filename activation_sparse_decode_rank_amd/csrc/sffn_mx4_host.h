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

// Whether the workgroups of a product hold the M rows of x in their LDS, codes and scales: every one
// of them does it for all rows, so few of them, and within the LDS that leaves two workgroups a
// compute unit. Float rows are held in 4-bit blocks on the way. 4 rows x 4096 x 4096 take 4.9 us so,
// 5.8 split over a tile's waves; 8 rows 6.5 and 5.8 (1 x 12288 x 49152: 49 and 63 us).
constexpr int kMx4FewRows = 4;
constexpr size_t kMx4FewLds = 48 * 1024;
inline size_t mx4_few_lds(size_t M, int K) { return M * (size_t)mx4_padded(K) * 17; }
inline bool mx4_few(size_t M, int K) {
  return M <= (size_t)kMx4FewRows && mx4_few_lds(M, K) <= kMx4FewLds;
}

// The kernel that M rows and N channels of nb blocks take: the one with the least time by a fit of
// measured ones, in microseconds: a + (b + (f - b) l) k for tiles that fill a share l of the device's
// room for them at once, k thousands of values long, and a + f k for each full room before them.
enum Mx4Form {
  kMx4Few, kMx4Split16, kMx4Split16x32, kMx4Split32, kMx4Split64, kMx4Tile64, kMx4Tile64x128, kMx4Tile128,
  kMx4Tile256
};
inline int mx4_form(size_t M, size_t N, int nb) {
  struct Fit {
    int form;
    size_t ch, tk, room;
    double a, b, f;
  };
  static const Fit fits[] = {{kMx4Split16, 16, 16, 512, 2.2, 0.36, 0.57},
                             {kMx4Split16x32, 16, 32, 512, 2.4, 0.38, 0.76},
                             {kMx4Split32, 32, 32, 512, 2.6, 0.48, 0.97},
                             {kMx4Split64, 64, 64, 256, 3.7, 0.69, 1.18},
                             {kMx4Tile64, 64, 64, 1024, 3.0, 1.9, 5.4},
                             {kMx4Tile64x128, 64, 128, 512, 6.0, 1.9, 3.5},
                             {kMx4Tile128, 128, 128, 512, 7.0, 2.65, 5.1},
                             {kMx4Tile256, 256, 256, 256, 9.0, 4.6, 8.6}};
  if (mx4_few(M, nb * 32)) return kMx4Few;
  const double k = nb / 32.0;
  int best = kMx4Tile256;
  double least = 1e300;
  for (const Fit& t : fits) {
    const size_t tiles = ((M + t.tk - 1) / t.tk) * ((N + t.ch - 1) / t.ch);
    const size_t full = (tiles - 1) / t.room;
    const double l = (double)(tiles - full * t.room) / (double)t.room;
    const double us = (double)full * (t.a + t.f * k) + t.a + (t.b + (t.f - t.b) * l) * k;
    if (us < least) {
      least = us;
      best = t.form;
    }
  }
  return best;
}

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
