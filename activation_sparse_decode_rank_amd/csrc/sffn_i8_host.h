// Host-side planning of the 8-bit products and the expert layer: pure C++ with no HIP
// dependency, so that it can be built and checked on its own.
#pragma once
#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace sffn {
namespace host {

inline size_t up_to(size_t v, size_t m) { return (v + m - 1) / m * m; }

// 8-bit rows of activations are padded with zeros to whole blocks of the products (256 bytes);
// the products read them up to a multiple of 128 bytes.
constexpr int kI8Step = 256;
constexpr int kI8Read = 128;
inline int i8_kpad(int K) { return (int)up_to((size_t)K, kI8Step); }

// Rows of a product tile, from the mean rows of a group (of the whole product where there are
// no groups) and the rows of w. Up to 32 the weights are streamed past them; above, the largest
// tile that still gives the device's 256 compute units (half of it, at most, idle at the end) two
// rounds of work, since larger tiles read less.
inline int i8_tile(size_t rows, size_t groups, size_t rows_w) {
  const size_t mean = (rows + groups - 1) / groups;
  if (mean <= 32) return mean <= 16 ? 16 : 32;
  auto tiles = [&](size_t t, size_t ch) {
    return groups * ((mean + t - 1) / t) * ((rows_w + ch - 1) / ch);
  };
  if (mean > 192 && tiles(256, 256) >= 512) return 256;
  if (mean > 96 && tiles(128, 256) >= 512) return 128;
  return 64;
}

// most rows, channels or columns of one call: they are rounded up to tiles in 32 bits
constexpr int kI8MaxCount = INT32_MAX - 1023;  // 2^31 - 1024

// Whether the tiles of M rows and N channels fit one launch, of less than 2^32 threads. Up to 32
// rows the grid goes by the device instead.
inline bool i8_launches(size_t M, size_t N) {
  const size_t t = (size_t)i8_tile(M, 1, N);
  if (t <= 32) return true;
  const size_t ch = t == 64 ? 128 : 256, threads = t == 64 ? 256 : 512;  // 64 channels: few tiles only
  return (((M + t - 1) / t) * ((N + ch - 1) / ch) + 8) * threads < (size_t)1 << 32;
}

// Whether M rows of K values are held in 8 bits by the product itself: every workgroup does it
// for all rows, so few of them, and within the LDS that leaves two workgroups a compute unit.
constexpr int kFusedRows = 4;
constexpr int kFusedLds = 64 * 1024;
inline bool i8_fused(size_t M, int K) {
  return M <= (size_t)kFusedRows && M * (size_t)i8_kpad(K) <= (size_t)kFusedLds;
}
// Whether one token of k slots goes through its experts in two launches, the slots' rows of f
// values held in LDS.
inline bool token_fused(int d, int f, int k) {
  return i8_fused(1, d) && (size_t)k * (size_t)i8_kpad(f) <= (size_t)kFusedLds;
}

// Scratch of an 8-bit product whose activations have to be held in 8 bits (or padded) first:
// the rows, then their scales.
struct I8MatmulCarve {
  size_t q, scale, bytes;
};
inline I8MatmulCarve i8_matmul_carve(size_t M, int K) {
  I8MatmulCarve c{};
  c.q = 0;
  c.scale = up_to(M * (size_t)i8_kpad(K), 256);
  c.bytes = c.scale + up_to(M * 4, 256);
  return c;
}

// most tiles that `rows` sorted rows of E experts can make
inline size_t experts_max_tiles(size_t rows, size_t E, int tile) {
  return rows / (size_t)tile + std::min(rows, E);
}

// Scratch of the expert layer for a chunk of T tokens of k slots each (R = T k rows).
struct ExpertsCarve {
  size_t xq, xs;        // the tokens in 8 bits [T][i8_kpad(d)] and their scales
  size_t offs, src;     // sorted rows: first of each expert [E + 1], slot of each row [R]
  size_t tiles, count;  // tile table [max_tiles] of (expert, first row), number of tiles
  size_t h, hq, hs;     // activations fp32 [R][ldh], 8 bits [R][i8_kpad(f)], scales [R]
  size_t part;          // down product of each slot fp32 [R][ldp]
  size_t ldh, ldp;
  int tile, max_tiles;
  size_t bytes;
};
inline ExpertsCarve experts_carve(int E, int d, int f, size_t T, size_t k) {
  ExpertsCarve c{};
  const size_t R = T * k;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += up_to(bytes, 256);
    return at;
  };
  c.tile = i8_tile(R, std::min(R, (size_t)E), (size_t)std::min(f, d));
  c.max_tiles = (int)experts_max_tiles(R, (size_t)E, c.tile);
  c.ldh = up_to((size_t)f, 64);
  c.ldp = up_to((size_t)d, 64);
  c.xq = take(T * (size_t)i8_kpad(d));
  c.xs = take(T * 4);
  c.offs = take(((size_t)E + 1) * 4);
  c.src = take(R * 4);
  c.tiles = take(experts_max_tiles(R, (size_t)E, 16) * 8);  // the most any tile makes
  c.count = take(4);
  c.h = take(R * c.ldh * 4);
  c.hq = take(R * (size_t)i8_kpad(f));
  c.hs = take(R * 4);
  c.part = take(R * c.ldp * 4);
  c.bytes = o;
  return c;
}

// Most rows one chunk may have, and most tokens: the rows' and the sums' launches stay below 2^32
// threads (1024 a token at most where it is held in 8 bits, 256 for each 1024 channels of its sum).
constexpr size_t kExpertsMaxRows = (size_t)1 << 21;
inline size_t experts_max_tokens(int d, int k) {
  const size_t blocks = ((size_t)d + 1023) / 1024;
  return std::max<size_t>(1, std::min(kExpertsMaxRows / (size_t)k, ((size_t)1 << 23) / blocks));
}
// The products reach up to 32 rows of w with 32-bit offsets.
constexpr int64_t kI8MaxLd = (int64_t)1 << 24;

// tokens per chunk that work_bytes holds (0: not even one), at most T
inline int experts_chunk(int E, int d, int f, int T, int k, size_t work_bytes) {
  size_t lo = 0, hi = std::min((size_t)T, experts_max_tokens(d, k));
  while (lo < hi) {
    const size_t mid = (lo + hi + 1) / 2;
    if (experts_carve(E, d, f, mid, (size_t)k).bytes <= work_bytes)
      lo = mid;
    else
      hi = mid - 1;
  }
  return (int)lo;
}

// The chunks of a call of T tokens, `size` tokens each but the last. 64 bits: the last one's end
// may pass 32.
struct Chunks {
  int64_t T, size, count;
  Chunks(int T_, int size_) : T(T_), size(size_), count((T + size - 1) / size) {}
  int64_t first(int64_t i) const { return i * size; }
  int tokens(int64_t i) const { return (int)std::min(size, T - first(i)); }
};

// The order in which chunks can go whose outputs may lie over inputs: a chunk reads its rows of x
// before it writes its rows of y, so no y row may meet an x row of a chunk that comes after its
// own. Rows of x: xb bytes, xp apart from x on; rows of y likewise.
enum class ChunkOrder { Forward, Backward, None };
inline ChunkOrder chunk_order(const Chunks& c, uintptr_t x, int64_t xp, int64_t xb, uintptr_t y,
                              int64_t yp, int64_t yb) {
  typedef __int128 I;
  const I T = c.T, at = (I)x - (I)y;  // bytes from y on: x's row t at at + t xp, y's at t yp
  if (c.count == 1 || at >= (T - 1) * yp + yb || at + (T - 1) * xp + xb <= 0) return ChunkOrder::Forward;
  auto floor_div = [](I a, I b) { return a >= 0 ? a / b : -((-a + b - 1) / b); };
  bool later = false, earlier = false;  // a y row meets an x row of a later (an earlier) chunk
  if (xp == yp) {  // the y rows that meet x's row t are t + lo .. t + hi, for every t
    const I lo = floor_div(at - yb, yp) + 1, hi = floor_div(at + xb - 1, yp);
    later = lo <= -1 && std::min<I>(hi, -1) > -T && lo <= hi;
    earlier = hi >= 1 && std::max<I>(lo, 1) < T && lo <= hi;
  } else {
    for (int64_t t = 0; t < c.T && !(later && earlier); ++t) {
      const I lo = std::max<I>(floor_div(at + t * (I)xp - yb, yp) + 1, 0);
      const I hi = std::min<I>(floor_div(at + t * (I)xp + xb - 1, yp), T - 1);
      if (lo > hi) continue;
      later |= lo / c.size < t / c.size;
      earlier |= hi / c.size > t / c.size;
    }
  }
  return !later ? ChunkOrder::Forward : !earlier ? ChunkOrder::Backward : ChunkOrder::None;
}

}  // namespace host
}  // namespace sffn
