// paged.cuh — what the kernels of the attention over the paged cache share: the list of tiles
// that the CTAs divide among themselves, look-ups in the page table, and small helpers.
#pragma once
#include "common.cuh"
#include "kernels.h"
#include "mma.cuh"

namespace dsmoe {
namespace paged {

constexpr float kNegInf = -INFINITY;
constexpr float kSlack = 8.f;   // log2 by which a score may exceed the row's reference

struct PagedArgs {
  int B, R, Hq, G, M, max_pages;
  int tile_log;     // log2 of the tokens of a tile
  int begin;        // places in the list before a (sequence, key head)'s tiles
  float scale_log2;
  const uint16_t* q;
  CacheView c;
  const int32_t* table;
  const int32_t* lengths;
  uint16_t* out;
  uint32_t* status;
  float* part_o;    // [2 grid][M][D]
  float* part_ml;   // [2 grid][M][2]
  int* span;        // [B][key heads][2]: the CTAs that begin and end a (sequence, head)
  int grid;         // CTAs that share the tiles
  bool pieces;      // all results are left as sums in the workspace, for another kernel's join
  unsigned long long* ready;   // (pieces) in the workspace's header: see began()
  unsigned long long call;     // (pieces) a number of this call's, never 0
};

// For the grid behind this one (PagedArgs::pieces), which may start now. That grid reads what the caller
// gives, but nothing of this one, so it need not wait for this one's end; yet what the grids before
// wrote is promised to be visible only to a grid that has waited itself, or to one that acquires
// what a thread released that had. So the call's number is released here, behind this grid's wait, and
// the next one waits after all if it does not find it (given_is_there). By one thread of a CTA.
// (Waiting always: 64 x 6 rows after 16k tokens 129.5 us against 124.5, 4 x 1 after 1000 19.9 against 17.4.)
__device__ __forceinline__ void began(const PagedArgs& a) {
  if (blockIdx.x == 0)
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(a.ready), "l"(a.call) : "memory");
  pdl_trigger();
}
// Whether it is released. (The last kernel of a call takes it back, so that a replay of a captured call
// does not find its predecessor's; a workspace may hold anything at first, but hardly this number.)
__device__ __forceinline__ bool given_is_there(const PagedArgs& a) {
  unsigned long long found;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(found) : "l"(a.ready) : "memory");
  return found == a.call;
}

// Where a CTA leaves its sums of a (sequence, key head): slot 0 when the run began before this CTA,
// slot 1 when it begins here and goes on in the next; `all` of it: behind those of the CTAs
// (PagedArgs::pieces only).
__device__ __forceinline__ int64_t piece_at(const PagedArgs& a, int b, int h, bool begins, bool all) {
  return all ? 2 * (int64_t)a.grid + (int64_t)b * a.c.heads + h
             : 2 * (int64_t)blockIdx.x + (begins ? 1 : 0);
}

// paged_few.cu: tiles of 64 tokens, up to 32 query rows per key head.
constexpr int kFewMaxRows = 32;
int few_ctas_per_sm(int M, int D, bool q8);
cudaError_t launch_few(const PagedArgs& p, int D, cudaStream_t s);

// paged_tc.cu: tiles of 128 tokens, one CTA per SM. The most query rows per key head: tensor
// memory holds S, O and two buffers of the sums, 4 N columns of 512 (and up to 96 rows a second
// buffer of S, up to 64 columns of O for either part of P).
constexpr int kTcMaxRows = 128;
cudaError_t launch_tc(const PagedArgs& p, int D, cudaStream_t s);

// paged_attn.cu: the kernel of a call alone, every (sequence, key head) left as pieces in the
// workspace (of pieces_workspace() bytes, the header first) for the caller's join. *args: what
// the kernel was given.
size_t pieces_workspace(const PagedAttnProblem& p);
cudaError_t launch_pieces(const PagedAttnProblem& p, uint8_t* ws, cudaStream_t s, PagedArgs* args);

__device__ __forceinline__ uint32_t smem_at(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The int8 values at bytes 0 and 2 of w as a bf16 pair, exactly: (128 + low 7 bits) minus
// 128 or, with the sign bit, 256.
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  uint32_t m, c, d;
  asm("lop3.b32 %0, %1, 0x007F007F, 0x43004300, 0xEA;" : "=r"(m) : "r"(w));
  asm("lop3.b32 %0, %1, 0x00800080, 0x43004300, 0xEA;" : "=r"(c) : "r"(w));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(c));
  return d;
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x2_t(uint32_t addr, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
               : "=r"(r0), "=r"(r1)
               : "r"(addr)
               : "memory");
}
// Byte offset of 16-byte chunk c of row r in a tile of rows of RB bytes: the eight rows of
// an ldmatrix meet eight different bank groups.
template <int RB>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if constexpr (RB == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  return r * RB + ((c ^ (r & 7)) << 4);
}

__device__ __forceinline__ int seq_len(const PagedArgs& a, int b) {
  const int n = a.lengths[b], cap = a.max_pages << a.c.page_shift;
  return n < 0 ? 0 : (n > cap ? cap : n);
}
__device__ __forceinline__ int tiles_of(const PagedArgs& a, int len) {
  return (len + (1 << a.tile_log) - 1) >> a.tile_log;
}

// The list of tiles: sequences, then key heads, then tiles along the length. Beginning and
// ending a (sequence, key head) costs about as much as `begin` tiles, so each non-empty one
// takes that many positions before its tiles, and the CTAs share the positions evenly.
__device__ __forceinline__ int places_of(const PagedArgs& a, int tiles) {
  return tiles ? tiles + a.begin : 0;
}

// The place of a tile in the list.
struct Cursor {
  int b, h, tile, tiles, len;
  __device__ __forceinline__ void open(const PagedArgs& a) {   // first non-empty from b on
    for (; b < a.B; ++b) {
      len = seq_len(a, b);
      tiles = tiles_of(a, len);
      if (tiles) break;
    }
  }
  __device__ __forceinline__ void next(const PagedArgs& a) {
    if (++tile < tiles) return;
    tile = 0;
    if (++h < a.c.heads) return;
    h = 0;
    ++b;
    open(a);
  }
};

// CTAs that share `total` positions: every one has some.
__device__ __forceinline__ int64_t cta_count(const PagedArgs& a, int64_t total) {
  return total < a.grid ? total : a.grid;
}
// Notes that this CTA has the first or the last tile of a (sequence, key head).
__device__ __forceinline__ void note_span(const PagedArgs& a, const Cursor& at, bool begins,
                                          bool ends) {
  int* const span = a.span + 2 * ((int64_t)at.b * a.c.heads + at.h);
  if (begins) span[0] = blockIdx.x;
  if (ends) span[1] = blockIdx.x;
}

// The run of tiles of CTA `cta`: its first tile's cursor and the number of tiles (0: none).
// All lanes of a warp together.
__device__ __forceinline__ int cta_run(const PagedArgs& a, int cta, int lane, Cursor* cur) {
  // lengths of the first 32 sequences stay in registers, the others are read again
  const int len0 = lane < a.B ? seq_len(a, lane) : 0;
  int64_t sum = places_of(a, tiles_of(a, len0));
  for (int b0 = 32; b0 < a.B; b0 += 32)
    sum += b0 + lane < a.B ? places_of(a, tiles_of(a, seq_len(a, b0 + lane))) : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int64_t total = sum * a.c.heads, ctas = cta_count(a, total);
  if (cta >= ctas) return 0;
  const int64_t ends[2] = {cta * total / ctas, (cta + 1) * total / ctas};
  // the tiles before each end: positions less those that are no tiles
  int64_t tiles_before[2] = {0, 0};
  int64_t before = 0, pairs = 0;   // positions and non-empty sequences, per key head
  bool found[2] = {false, false};
  for (int b0 = 0; b0 < a.B && !(found[0] && found[1]); b0 += 32) {
    const int len = b0 == 0 ? len0 : (b0 + lane < a.B ? seq_len(a, b0 + lane) : 0);
    const int tiles = tiles_of(a, len), mine = places_of(a, tiles);
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const unsigned filled = __ballot_sync(0xffffffffu, mine > 0);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const unsigned past = __ballot_sync(0xffffffffu, (before + upto) * a.c.heads > ends[e]);
      if (found[e] || !past) continue;
      found[e] = true;
      const int l = __ffs(past) - 1;
      const int places = __shfl_sync(0xffffffffu, mine, l);
      const int64_t first = (before + __shfl_sync(0xffffffffu, upto, l) - places) * a.c.heads;
      const int h = (int)((ends[e] - first) / places), pos = (int)((ends[e] - first) % places);
      const int64_t begun = (pairs + __popc(filled & ((1u << l) - 1))) * a.c.heads + h;
      tiles_before[e] = ends[e] - begun * a.begin - (pos < a.begin ? pos : a.begin);
      const int n = __shfl_sync(0xffffffffu, tiles, l), ln = __shfl_sync(0xffffffffu, len, l);
      if (e == 0) *cur = Cursor{b0 + l, h, pos > a.begin ? pos - a.begin : 0, n, ln};
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
    pairs += __popc(filled);
  }
  if (!found[1]) tiles_before[1] = total - pairs * a.c.heads * a.begin;   // the end of the list
  return (int)(tiles_before[1] - tiles_before[0]);
}
// Page of token t of sequence b of `len` tokens, or -1: no such token, or a bad table entry.
__device__ __forceinline__ int page_of(const PagedArgs& a, int b, int t, int len) {
  if (t >= len) return -1;
  const int p = a.table[(int64_t)b * a.max_pages + (t >> a.c.page_shift)];
  return p >= 0 && p < a.c.pages ? p : -1;
}

}  // namespace paged
}  // namespace dsmoe
