// prefix.cuh — what the kernel of the shared prefixes and its join agree on: the list of tiles, its
// division among the CTAs, and where the sums are left.
//
// All query rows of a prefix's sequences for one key head are the M dimension of one product with the
// prefix's keys. They come in tiles of 128 rows, two of which make a unit; the last unit of an odd
// number has one. The list: prefixes, then key heads, then units, then tiles of 128 tokens. A CTA
// works on the two row tiles of a unit with every token tile, or, in a unit of one row tile, on
// two token tiles with the same rows, so that it always has two streams of scores. Positions in the
// list are (row tile, token tile) pairs, behind `kBegin` for what beginning and ending a unit
// costs; the CTAs share the positions evenly.
#pragma once
#include "paged_tc.cuh"

namespace dsmoe {
namespace prefix {

using namespace paged;

constexpr int kTok = 128;      // tokens of a tile
constexpr int kRows = 128;     // query rows of a tile
constexpr int kBegin = 2;

struct PrefixArgs {
  PagedArgs own;        // the sequences' own tokens; queries, cache, results
  int P, per;           // prefixes; sequences of each
  int MP;               // query rows of a prefix per key head
  uint32_t m_inverse;   // 2^32 / own.M, rounded up (M = 1: 0, for 2^32)
  int tiles, units;     // row tiles and units of a prefix per key head
  int rows;             // of a piece: 128, or MP
  int max_pages;        // of a prefix
  const int32_t* table;
  const int32_t* lengths;
  int grid;
  int* span;            // [units of all][2]: the CTAs that begin and end a unit
  float* part_o;        // [units of all + grid][2][rows][D]
  float* part_ml;       // [units of all + grid][2][rows][2]
};

__device__ __forceinline__ int prefix_len(const PrefixArgs& a, int p) {
  const int n = a.lengths[p], cap = a.max_pages << a.own.c.page_shift;
  return n < 0 ? 0 : (n > cap ? cap : n);
}
__device__ __forceinline__ int token_tiles(int len) { return (len + kTok - 1) / kTok; }
// Positions of a prefix's head.
__device__ __forceinline__ int64_t head_places(const PrefixArgs& a, int T) {
  return T ? (int64_t)a.tiles * T + (int64_t)a.units * kBegin : 0;
}
// Row tiles of a unit.
__device__ __forceinline__ int unit_tiles(const PrefixArgs& a, int u) {
  return 2 * u + 1 < a.tiles ? 2 : 1;
}
// n / own.M of a row number n < 2^19 (the rounding of the inverse adds less than 2^19 x 2^7 / 2^32).
__device__ __forceinline__ unsigned over_m(const PrefixArgs& a, unsigned n) {
  return a.m_inverse ? __umulhi(n, a.m_inverse) : n;
}
// Positions of the whole list, given the length of prefix `lane`. All lanes of a warp together.
__device__ __forceinline__ int64_t list_places(const PrefixArgs& a, int lane, int len) {
  int64_t sum = lane < a.P ? head_places(a, token_tiles(len)) : 0;
  for (int p = lane + 32; p < a.P; p += 32) sum += head_places(a, token_tiles(prefix_len(a, p)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum * a.own.c.heads;
}
// CTAs that share them, three positions or more each: so a CTA between those that begin and end a
// unit has some of its tiles.
__device__ __forceinline__ int64_t list_ctas(const PrefixArgs& a, int64_t total) {
  return total < 3 * (int64_t)a.grid ? total / 3 : a.grid;   // (a unit has three at least)
}
// The token tile that position x of a unit of w row tiles belongs to: where a CTA begins there, the
// first it takes; where it ends, the first it leaves.
__device__ __forceinline__ int tile_at(int64_t x, int w) {
  return x < kBegin ? 0 : (int)(x - kBegin) >> (w - 1);
}
// Where CTA `cta` leaves its sums of a unit, counted over all: CTAs and units only ever go up along
// the list, so no two pairs have the same sum.
__device__ __forceinline__ int64_t unit_piece(const PrefixArgs& a, int p, int h, int u, int cta) {
  return ((int64_t)p * a.own.c.heads + h) * a.units + u + cta;
}

// A stretch of a unit's token tiles.
struct Run {
  int p, h, u, w, len, t0, t1;
};

// Walks a CTA's runs.
struct Walk {
  int64_t pos, end, start;   // start: of the head that pos is in
  int p, h, len, T;
  // All lanes of a warp together.
  // (len: prefix_len() of prefix `lane`)
  __device__ __forceinline__ void open(const PrefixArgs& a, int cta, int lane, int lane_len) {
    const int64_t total = list_places(a, lane, lane_len), ctas = list_ctas(a, total);
    pos = end = 0;
    if (cta >= ctas) return;
    // (the first total % ctas have one more)
    const int64_t each = total >> 32 ? total / ctas : (unsigned)total / (unsigned)ctas;
    const int64_t more = total - each * ctas;
    pos = cta * each + (cta < more ? cta : more);
    end = pos + each + (cta < more ? 1 : 0);
    start = 0;
    p = -1;
    skip(a);
    for (;;) {   // the prefix
      const int64_t n = head_places(a, T) * a.own.c.heads;
      if (pos < start + n || pos == end) break;
      start += n;
      skip(a);
    }
    const int64_t per_head = head_places(a, T);
    h = (int)__fdividef((float)(pos - start), (float)per_head);   // (below 256, off by one at most)
    if (h * per_head > pos - start) --h;
    if ((h + 1) * per_head <= pos - start) ++h;
    start += h * per_head;
  }
  __device__ __forceinline__ void skip(const PrefixArgs& a) {   // to the next prefix with tokens
    h = 0;
    do {
      ++p;
      len = p < a.P ? prefix_len(a, p) : 0;
      T = token_tiles(len);
    } while (T == 0 && p < a.P);
    if (p >= a.P) end = pos;   // (it is, unless the lengths change under the kernel)
  }
  __device__ __forceinline__ bool next(const PrefixArgs& a, Run* r) {
    while (pos < end) {
      // (a head's positions fit 31 bits: up to 4096 row tiles of up to 2^17 token tiles)
      const unsigned x = (unsigned)(pos - start), full = 2u * T + kBegin;
      const int u = (int)(x / full);
      const int w = unit_tiles(a, u);
      const int64_t first = start + (int64_t)u * full, behind = first + (int64_t)w * T + kBegin;
      *r = Run{p, h, u, w, len, tile_at(pos - first, w), end >= behind ? T : tile_at(end - first, w)};
      if (end < behind) {
        pos = end;
      } else {
        pos = behind;
        if (u + 1 == a.units) {
          start = behind;
          if (++h == a.own.c.heads) skip(a);
        }
      }
      if (r->t1 > r->t0) return true;
    }
    return false;
  }
};

// prefix_tc.cu
cudaError_t launch_prefix_tc(const PrefixArgs& a, int D, cudaStream_t s);

}  // namespace prefix
}  // namespace dsmoe
