// What the paged-cache kernels share: how a batch's new rows, positions and
// pages are read, and which tokens a row sees.
//
// A resident layer keeps its rows in pages of a pool: token t of sequence b is
// slot page_table[b][t / page_size] * page_size + t % page_size. A step brings
// rows row0[b] .. row0[b+1]-1 of sequence b, the last ones of its seq_len[b]
// tokens: its row i is at position seq_len[b] - n + i and sees tokens t <=
// position (with a window: those with t > position - window, or t < n_sink).
// Everything read from the device is clamped to the host's bounds, so no table
// or length, however wrong, leads outside a buffer.
#pragma once

#include "common.hpp"

namespace {

constexpr int kPagedRow = 576;             // values per row (key width)
constexpr int kPagedVal = 512;             // value width: the row's first values
constexpr int kPagedChunks = kPagedRow * 2 / 16;   // 16-byte pieces of a row (72)

struct Pages {
  const int32_t* table;   // [B, ld]
  int64_t ld;             // page-table entries per sequence
  uint32_t n_slots;       // rows in the pool
  uint32_t n_pages;       // pages that begin in the pool
  int size;               // tokens per page
  uint32_t mul;           // t / size = (mulhi(t, mul) + t) >> shift for t < 2^31
  int shift;
};

inline Pages make_pages(const int32_t* table, int64_t ld, int64_t n_slots, int size) {
  int l = 0;
  while ((1u << l) < (uint32_t)size) ++l;                  // ceil(log2 size), size <= 2^20
  const uint64_t mul = (((1ull << l) - (uint64_t)size) << 32) / (uint64_t)size + 1;
  return Pages{table, ld, (uint32_t)n_slots, (uint32_t)((n_slots + size - 1) / size), size, (uint32_t)mul, l};
}

__device__ __forceinline__ uint32_t page_index(const Pages& pg, int t) {
  return (__umulhi((uint32_t)t, pg.mul) + (uint32_t)t) >> pg.shift;
}

// Slot of the token `off` tokens into page `page`, or -1 where that is none of
// the pool's.
__device__ __forceinline__ int slot_in(const Pages& pg, int page, int off) {
  const uint32_t s = (uint32_t)page * (uint32_t)pg.size + (uint32_t)off;   // < 2^31 + 2^20 for a page of the pool
  return (uint32_t)page < pg.n_pages && s < pg.n_slots ? (int)s : -1;
}

// Slot of token t of the sequence whose page-table row is `row`, or -1 where
// the table has no valid page for it.
__device__ __forceinline__ int slot_of(const Pages& pg, const int32_t* row, int t) {
  const uint32_t idx = page_index(pg, t);
  if ((int64_t)idx >= pg.ld) return -1;
  return slot_in(pg, row[idx], t - (int)idx * pg.size);
}

// The new rows of one sequence, clamped: rows [first, first + n), row i at
// position pos0 + i (negative: it sees nothing), tokens below len exist.
struct SeqRows {
  int first, n, pos0, len;
};

__device__ __forceinline__ SeqRows seq_rows(const int32_t* row0, const int32_t* seq_len, const Pages& pg, int b, int T,
                                            int max_rows, int max_len) {
  const int r0 = min(max(row0[b], 0), T), r1 = min(max(row0[b + 1], r0), T);
  const int64_t cap = min((int64_t)max_len, pg.ld * (int64_t)pg.size);
  const int len = (int)min((int64_t)max(seq_len[b], 0), cap);
  return SeqRows{r0, min(r1 - r0, max_rows), len - (r1 - r0), len};
}

// Inclusive prefix sum over the wave's lanes in the vector unit (rows of 16 by
// shifts, then the rows' last lanes to the rows behind them), and the last
// lane's value, the same in every lane.
__device__ __forceinline__ int lanes_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);   // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);   // row_bcast 15 to rows 1, 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);   // row_bcast 31 to rows 2, 3
  return x;
}
__device__ __forceinline__ int last_lane(int x) { return __builtin_amdgcn_readlane(x, 63); }

// What a workgroup does: span sp of the n_span spans of tile mt of sequence b
// (-1: nothing), whose new rows are sr; in a plan, the batch's tile `tile` of
// `tiles`.
struct Work {
  int b, mt, sp, n_span;
  SeqRows sr;
  int tile, tiles;
};
__device__ __forceinline__ SeqRows rows_of_lane(const SeqRows& sr, int l) {
  return SeqRows{__builtin_amdgcn_readlane(sr.first, l), __builtin_amdgcn_readlane(sr.n, l),
                 __builtin_amdgcn_readlane(sr.pos0, l), __builtin_amdgcn_readlane(sr.len, l)};
}

// Tile `tile` of the batch as one piece of work, when sequence b's n rows of H
// heads make ceil(n H / per) tiles and the tiles are numbered through the
// batch. Every lane of the wave takes part: 64 sequences a round.
__device__ __forceinline__ Work tile_work(const int32_t* row0, const int32_t* seq_len, const Pages& pg, int B, int T,
                                          int H, int max_rows, int max_len, int per, int tile) {
  const int lane = ech::lane_id();
  int base = 0;
  for (int b0 = 0; b0 < B; b0 += 64) {
    const int b = b0 + lane;
    SeqRows sr{0, 0, 0, 0};
    if (b < B) sr = seq_rows(row0, seq_len, pg, b, T, max_rows, max_len);
    const int tiles = (sr.n * H + per - 1) / per;          // T H < 2^30
    const int incl = lanes_scan(tiles);
    const unsigned long long past = __ballot(base + incl > tile);
    if (past != 0ull) {
      const int l = __builtin_ctzll(past);
      const int before = __builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(tiles, l);
      return Work{b0 + l, tile - base - before, 0, 1, rows_of_lane(sr, l), 0, 0};
    }
    base += last_lane(incl);
  }
  return Work{-1, 0, 0, 1, SeqRows{0, 0, 0, 0}, 0, 0};
}

// Whether a row at position p sees token t (t < len is the caller's).
__device__ __forceinline__ bool sees(int p, int t, int window, int n_sink) {
  return t <= p && (window == 0 || t > p - window || t < n_sink);
}

inline bool aligned16_(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Host checks shared by the entry points.
inline bool pages_ok(int64_t n_slots, int page_size, const int32_t* table, int64_t ld) {
  return table && n_slots >= 1 && n_slots < (1ll << 31) && page_size >= 1 && page_size <= (1 << 20) && ld >= 1 &&
         ld < (1ll << 31);
}
inline bool batch_ok(int B, int T, int max_rows, int max_len) {
  return B >= 1 && B <= 65535 && T >= 0 && max_rows >= 0 && max_len >= 0 && max_len <= (1 << 30);
}

}  // namespace
