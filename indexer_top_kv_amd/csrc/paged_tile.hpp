// What the matrix-core kernels over paged rows share: operand types, the step
// layout in LDS, the ranges of tokens that a tile of queries reads, and the
// split of tiles over the CUs.
#pragma once

#include "paged.hpp"

namespace {

typedef __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16 bf16x8_t;
typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16_t;
typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 bf16x4_t;
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef short v4s_t __attribute__((ext_vector_type(4)));
typedef short v8s_t __attribute__((ext_vector_type(8)));

constexpr int kStepTok = 32;                 // tokens per step
constexpr int kKs16 = kPagedRow / 16;        // contraction steps of the scores (36)
constexpr int kVPitch = kPagedVal * 2 + 32;  // bytes per token of the value part in LDS (two spare pieces: banks)
constexpr int kTailAt = kStepTok * kVPitch;  // the rows' last 64 values (rotary part), 128 bytes a token
constexpr int kTileB = kTailAt + kStepTok * 128;
#define ECH_LDS_PTR(p) ((__attribute__((address_space(3))) void*)(p))

__device__ __forceinline__ bf16x8_t ld_bf16x8(const uint8_t* p) {
  return __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t*>(p));
}

__device__ __forceinline__ f32x16_t mfma32(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Maximum / sum over the two lanes (l, l ^ 32) that share a query.
__device__ __forceinline__ float pair_max(float x) {
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float pair_sum(float x) {
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// Direct-to-LDS loads of 1 KiB: lane l's 16 bytes go to lds + 16 l. From inline
// asm, so that the compiler does not wait for them before other LDS reads; they
// write no register, and the caller waits for them by count.
__device__ __forceinline__ void lds_load_row(uint32_t lds, uint32_t voff, const uint8_t* src) {   // src uniform
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(voff), "s"(src)
               : "memory", "m0");
}
__device__ __forceinline__ void lds_load_lanes(uint32_t lds, const uint8_t* src) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory", "m0");
}
__device__ __forceinline__ void lds_load_dwords(uint32_t lds, const void* src) {   // 4 bytes a lane
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(src) : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(ECH_LDS_PTR(const_cast<void*>(p))));
}

// The tokens a tile of queries at positions [p_lo, p_hi] reads, as up to two
// ranges: [0, n0) and [w0, w1). Steps of STEP tokens run through the first,
// then the second.
struct Ranges {
  int n0, w0, w1, s0, steps;
};
template <int STEP>
__device__ __forceinline__ Ranges ranges_of(int p_lo, int p_hi, int window, int n_sink) {
  const int end = p_hi + 1;                               // <= len
  const int w0 = window == 0 ? 0 : max(0, p_lo - window + 1);
  Ranges r;
  if (window == 0 || w0 <= n_sink) {                      // one range
    r = Ranges{0, 0, max(end, 0), 0, 0};
  } else {
    r = Ranges{min(n_sink, end), w0, end, 0, 0};
  }
  r.s0 = (r.n0 + STEP - 1) / STEP;
  r.steps = r.s0 + (r.w1 - r.w0 + STEP - 1) / STEP;
  return r;
}

// Bits of the tokens t0 .. t0 + 31 that a query at position p sees.
__device__ __forceinline__ uint32_t sees_bits(int p, int t0, int window, int n_sink) {
  const int d = p - t0;    // last visible, relative
  uint32_t bits = d < 0 ? 0u : (d >= 31 ? 0xffffffffu : (2u << d) - 1u);
  if (window != 0) {
    const int lo = d - window + 1, sk = n_sink - t0;
    const uint32_t win = lo <= 0 ? 0xffffffffu : (lo >= 32 ? 0u : 0xffffffffu << lo);
    const uint32_t first = sk <= 0 ? 0u : (sk >= 32 ? 0xffffffffu : (1u << sk) - 1u);
    bits &= win | first;
  }
  return bits;
}

constexpr int kCus = 256;
constexpr int kMinSpan = 4;          // steps a span is worth its start and its partial
constexpr int kPlanSeqs = 256;       // sequences a plan covers (four per lane)

// Whether a plan covers B sequences, and its sums, steps of so many tiles that
// read up to `tokens` each, stay in 31 bits (`tiles` whatever the row offsets say).
inline bool plan_fits(int B, int64_t tiles, int64_t tokens) {
  return B <= kPlanSeqs && tiles * (tokens / kStepTok + 1) < (1ll << 30);
}

__device__ __forceinline__ int lanes_max(int x) {           // x >= 0
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false));
  return last_lane(x);
}

// The batch's tiles split over the card's CUs: every tile takes ceil(steps /
// S) spans with one S for all, the smallest for which the spans are at most as
// many as the CUs, so that a batch of unequal lengths ends at one time.
// (Spans of equal number per sequence instead: 32 decoded tokens at 128 heads
// over 8K to 16K tokens 165 us, with this 153 us. A tile per CU, not split: 881
// us, and 12 chunks of 77 rows at 16 heads over up to 5K tokens 282 us against
// 73 us.) All tiles of a sequence
// count as its last and longest. Every wave computes it alike, a sequence (of
// each 64) per lane. ALL: one tile per sequence, over all of its tokens, new
// rows or none.
template <int PER, int STEP, bool ALL = false>
__device__ __forceinline__ Work plan_work(const int32_t* row0, const int32_t* seq_len, const Pages& pg, int B, int T,
                                          int H, int max_rows, int max_len, int window, int n_sink, int wg) {
  const int lane = ech::lane_id();
  int nt[kPlanSeqs / 64], st[kPlanSeqs / 64];
  SeqRows sr[kPlanSeqs / 64];
  int tiles = 0, total = 0, longest = 1;
#pragma unroll
  for (int c = 0; c < kPlanSeqs / 64; ++c) {
    nt[c] = 0;
    st[c] = 1;
    sr[c] = SeqRows{0, 0, 0, 0};
    if (c * 64 < B) {
      const int b = c * 64 + lane;
      if (b < B) sr[c] = seq_rows(row0, seq_len, pg, b, T, max_rows, max_len);
      if (ALL) {
        nt[c] = sr[c].len > 0;
        st[c] = max(1, (sr[c].len + STEP - 1) / STEP);
      } else {
        nt[c] = (sr[c].n * H + PER - 1) / PER;
        if (nt[c] > 0)
          st[c] = max(1, ranges_of<STEP>(sr[c].pos0 + (nt[c] - 1) * PER / H, sr[c].pos0 + sr[c].n - 1, window, n_sink).steps);
      }
      tiles += nt[c];
      total += nt[c] * st[c];
      if (nt[c] > 0) longest = max(longest, st[c]);
    }
  }
  tiles = last_lane(lanes_scan(tiles));
  total = last_lane(lanes_scan(total));
  longest = lanes_max(longest);
  // ceil(x / S) by a reciprocal and one correction, which is exact: no S tried is
  // below total / kCus, so no quotient is above kCus + 1
  auto parts = [](int x, int S, float inv) -> int {
    const int y = x + S - 1, n = (int)((float)y * inv), rest = y - n * S;
    return n + (rest >= S) - (rest < 0);
  };
  auto spans = [&](int S) -> int {
    const float inv = __builtin_amdgcn_rcpf((float)S);
    int n = 0;
#pragma unroll
    for (int c = 0; c < kPlanSeqs / 64; ++c)
      if (c * 64 < B) n += nt[c] * parts(st[c], S, inv);
    return last_lane(lanes_scan(n));
  };
  int lo = max(kMinSpan * kStepTok / STEP, (total + kCus - 1) / kCus), hi = max(lo, longest);   // spans(hi) = tiles <= kCus
  if (tiles < kCus) hi = min(hi, max(lo, total / (kCus - tiles) + 1));         // sum ceil(x) < sum x + tiles
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (spans(mid) <= kCus) hi = mid;
    else lo = mid + 1;
  }
  const float inv = __builtin_amdgcn_rcpf((float)hi);
  int base = 0, tile0 = 0;
#pragma unroll
  for (int c = 0; c < kPlanSeqs / 64; ++c) {
    if (c * 64 < B) {
      const int n = parts(st[c], hi, inv), mine = nt[c] * n;
      const int incl = lanes_scan(mine);
      const unsigned long long past = __ballot(base + incl > wg);
      if (past != 0ull) {
        const int l = __builtin_ctzll(past);
        const int in = wg - base - __builtin_amdgcn_readlane(incl, l) + __builtin_amdgcn_readlane(mine, l);
        const int ns = __builtin_amdgcn_readlane(n, l), mt = in / ns;
        tile0 += __builtin_amdgcn_readlane(lanes_scan(nt[c]) - nt[c], l);
        return Work{c * 64 + l, mt, in - mt * ns, ns, rows_of_lane(sr[c], l), tile0 + mt, tiles};
      }
      base += last_lane(incl);
      tile0 += last_lane(lanes_scan(nt[c]));
    }
  }
  return Work{-1, 0, 0, 1, SeqRows{0, 0, 0, 0}, 0, tiles};
}

// This workgroup's place in a plan of kCus: workgroups go to the 8 XCDs in turn,
// and the spans of a tile, and a sequence's tiles, which read the same queries
// and rows, share an XCD's cache. (12 chunks of 77 rows 72.7 us in the order of
// the grid, 71.5 with this; a window of 1024 31.4 and 31.1.)
__device__ __forceinline__ int plan_wg() { return (int)(blockIdx.x & 7) * (kCus / 8) + (int)(blockIdx.x >> 3); }

// How a tile's partials are joined: its first query and how many it has, and
// which workgroups hold its spans (n_span <= 1: nothing to join).
struct PartInfo {
  int64_t first;
  int queries, base, n_span, spare;
};
// Written by the workgroup (wg in the plan) of a tile's first span; the grid's first marks
// the entries past the last tile, up to `bound`. Call from all threads.
__device__ __forceinline__ void note_tile(PartInfo* info, const Work& wk, int wg, int64_t first, int queries, int bound) {
  if (blockIdx.x == 0)
    for (int x = wk.tiles + threadIdx.x; x < bound; x += blockDim.x) info[x] = PartInfo{0, 0, 0, 0, 0};
  if (wk.b >= 0 && wk.sp == 0 && threadIdx.x == 0 && wk.tile < bound)
    info[wk.tile] = PartInfo{first, queries, wg, wk.n_span, 0};
}

}  // namespace
