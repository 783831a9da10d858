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
// compute unit. Float rows are held in 4-bit blocks on the way. 4 rows x 4096 x 4096 take 5.5 us so,
// 6.0 with a launch for x's rows and split over a tile's waves; 8 rows 6.7 and 6.1; 4 rows x 11008 x
// 4096 10.2 both ways, 5 rows 11.7 and 10.3 (1 x 12288 x 49152: 51 and 69). Rows that are held already
// take it too, so that both give the same bits: 4 x 4096 x 4096 5.1 us, 3.5 split over a tile's waves,
// 4 x 11008 x 4096 7.6 and 7.7, 4 x 12288 x 49152 48 and 64.
constexpr int kMx4FewRows = 4;
constexpr size_t kMx4FewLds = 48 * 1024;
inline size_t mx4_few_lds(size_t M, int K) { return M * (size_t)mx4_padded(K) * 17; }
inline bool mx4_few(size_t M, int K) {
  return M <= (size_t)kMx4FewRows && mx4_few_lds(M, K) <= kMx4FewLds;
}

// Whether workgroups hold 16 rows of x each in their LDS, and a wave has a tile to itself: for more
// rows, of at most 512 values (one group), and few tiles. Float rows: 42 x 345 x 3475 (M x K x N) takes
// 4.0 us so, 5.5 with a launch for x's rows in front, and that launch costs the host 3 to 4 us; 445 x
// 469 x 552 4.0 and 5.7; 1024 x 512 x 1024 (4096 tiles) 5.6 and 6.7, 1224 x 375 x 949 (4620) 7.2 and
// 7.8, 1007 x 502 x 1332 (5292) 8.4 and 7.5; of two groups, 77 x 950 x 610, 5.9 and 5.3. Rows that are
// held already take it at the same sizes, so that both give the same bits: 33 x 162 x 3983 3.0 us, 3.2
// split over a tile's waves, 13 x 451 x 180 2.7 both ways, 1024 x 512 x 1024 4.8 and 4.4.
constexpr size_t kMx4ShortTiles = 4096;
inline bool mx4_short(size_t M, size_t N, int nb) {
  return nb <= kMx4Group && ((M + 15) / 16) * ((N + 15) / 16) <= kMx4ShortTiles;
}
// Whether a product of float rows holds them in 4-bit blocks itself, without scratch
inline bool mx4_own(size_t M, size_t N, int K) {
  return mx4_few(M, K) || mx4_short(M, N, mx4_blocks(K));
}

// The kernel that M rows and N channels of nb blocks take: the one with the least time by a fit of
// measured ones, in microseconds: a + (b + (f - b) l) k for tiles that fill a share l of the device's
// room for them at once (what 256 compute units hold), k thousands of values long, and a + f k for each
// full room before them. Over 330 random sizes of 5 to 4000 rows its choice takes 1.9% more than the
// fastest of them in the mean, 33% at most (profiles/mx4_plan.txt).
enum Mx4Form {
  kMx4Few, kMx4Short, kMx4Split16, kMx4Split16x32, kMx4Split32, kMx4Split64, kMx4Tile64, kMx4Tile64x128, kMx4Tile128,
  kMx4Tile256
};
struct Mx4Fit {
  int form;
  size_t ch, tk, room, threads;
  double a, b, f;
  // a launch holds less than 2^32 threads
  bool launches(size_t M, size_t N) const { return (tiles(M, N) + 8) * threads < (size_t)1 << 32; }
  size_t tiles(size_t M, size_t N) const { return ((M + tk - 1) / tk) * ((N + ch - 1) / ch); }
  double us(size_t M, size_t N, double k) const {
    const size_t t = tiles(M, N), full = (t - 1) / room;
    const double l = (double)(t - full * room) / (double)room;
    return (double)full * (a + f * k) + a + (b + (f - b) * l) * k;
  }
};
constexpr Mx4Fit kMx4Fits[] = {{kMx4Split16, 16, 16, 512, 512, 2.2, 0.36, 0.57},
                              {kMx4Split16x32, 16, 32, 512, 512, 2.4, 0.38, 0.76},
                              {kMx4Split32, 32, 32, 512, 512, 2.6, 0.48, 0.97},
                              {kMx4Split64, 64, 64, 256, 512, 3.7, 0.69, 1.18},
                              {kMx4Tile64, 64, 64, 1024, 256, 3.0, 1.9, 5.4},
                              {kMx4Tile64x128, 64, 128, 512, 256, 6.0, 1.9, 3.5},
                              {kMx4Tile128, 128, 128, 512, 256, 7.0, 2.65, 5.1},
                              {kMx4Tile256, 256, 256, 256, 512, 9.0, 4.6, 8.6}};
// Whether M rows and N channels fit a launch: the largest tiles' do
inline bool mx4_launches(size_t M, size_t N) { return kMx4Fits[7].launches(M, N); }
inline const Mx4Fit& mx4_best(size_t M, size_t N, double k) {
  const Mx4Fit* best = &kMx4Fits[7];
  for (const Mx4Fit& t : kMx4Fits)
    if (t.launches(M, N) && t.us(M, N, k) < best->us(M, N, k)) best = &t;
  return *best;
}
// Where the largest tiles leave their last room half empty, the channels of that room may do better
// with smaller ones, in a launch of their own: the first n1 channels take `form`, the others `rest`.
// 512 x 12288 x 49152 takes 208 us so (127 and 82 of them), 227 in one launch.
struct Mx4Plan {
  int form, rest;
  size_t n1;  // N: one launch
};
inline Mx4Plan mx4_plan(size_t M, size_t N, int nb) {
  if (mx4_few(M, nb * 32)) return {kMx4Few, kMx4Few, N};
  if (mx4_short(M, N, nb)) return {kMx4Short, kMx4Short, N};
  const double k = nb / 32.0;
  const Mx4Fit& one = mx4_best(M, N, k);
  Mx4Plan p{one.form, one.form, N};
  const size_t down = (M + one.tk - 1) / one.tk, full = one.tiles(M, N) / one.room;
  if (one.form != kMx4Tile256 || full == 0) return p;
  const size_t n1 = full * one.room / down * one.ch;
  if (n1 == 0 || n1 >= N) return p;
  const Mx4Fit& rest = mx4_best(M, N - n1, k);
  if (rest.form != kMx4Tile256 && one.us(M, n1, k) + rest.us(M, N - n1, k) < 0.95 * one.us(M, N, k)) {
    p.rest = rest.form;
    p.n1 = n1;
  }
  return p;
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
