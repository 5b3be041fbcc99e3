// Attention of a step's new rows over the pages of a resident cache
// (ech_paged_attn): a prompt's chunk, single decoded tokens, or a ragged mix,
// causal, optionally with a sliding window and a few first tokens that stay
// visible. Rows are absorbed-MLA rows shared by every head (576 bf16 values,
// the first 512 of them the value), so a sequence's (row, head) pairs are one
// list of queries against one list of keys, and a tile takes 128 of them
// whatever the number of heads.
//
//   s[m][t] = scale q[m] . k[t],  o[m] = sum_t softmax(s)[m][t] v[t]
//
// One pass over the tokens with a running maximum and sum per query (fp32,
// base 2). Per 32-token step and workgroup of four waves, on
// v_mfma_f32_32x32x16_bf16:
//   S^T[token][m] = K . Q^T     wave w: the 32 queries of row tile w, whose
//                               fragments stay in registers (144)
//   O^T[col][m]  += V^T . P^T   wave w: value columns 128 w .. +127 of all 128
//                               queries (256 accumulators)
// so a step's rows are read from LDS by every wave for the scores but only
// once for the values, and P (8 KiB, bf16) crosses between the waves through
// LDS. The weights enter the value product as bf16, rounded to nearest (2^-8
// of each weight at most; the output is rounded to bf16 as well), while the
// sum that divides them is fp32 over the unrounded weights.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "paged_tile.hpp"

namespace {

constexpr int kMT = 128;                     // queries per workgroup
constexpr int kBufs = 3;
constexpr int kPPitch = 80;                  // bytes per query of P in LDS (64 + 16: bank spread)
constexpr int kKD = 3;                       // key fragments in flight
constexpr int kSplit = 30;                   // products of a step's scores before the barrier that publishes P

// The same onto an accumulator that stays in accumulation registers (the
// output takes all 256 of them, so none is left for the compiler to choose).
// The compiler does not see that this is a matrix instruction, so other
// instructions that touch the accumulator stand behind mfma32_acc_done.
__device__ __forceinline__ void mfma32_acc(f32x16_t& d, bf16x8_t a, bf16x8_t b) {
  asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(d) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mfma32_acc_done() { asm volatile("s_nop 15\n\ts_nop 7"); }

// 8 tokens x this lane's column, from two transposed reads of 4 tokens.
__device__ __forceinline__ bf16x8_t ld_tr8(const uint8_t* p0, const uint8_t* p1) {
  const v4s_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s_t*)(p0));
  const v4s_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s_t*)(p1));
  const v8s_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8_t, v);
}

// Where a score that does not count is not finite, its row holds infinities or
// NaN, and 0 x inf is NaN: the step's values that are not finite become 0 before
// the value product. What that product would have made of them for the queries
// that do see them is put in by an indicator product: A = 1 where a value is not
// finite, B = 1 where the query sees the token, and NaN where the sum is not 0
// (a weight of its own is NaN already, or 0 beside a score of -inf).
__device__ __forceinline__ bf16x8_t not_finite(bf16x8_t v) {
  u32x4_t w = __builtin_bit_cast(u32x4_t, v);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = ((w[j] & 0x7f80u) == 0x7f80u ? 0x3f80u : 0u) | ((w[j] & 0x7f800000u) == 0x7f800000u ? 0x3f800000u : 0u);
  return __builtin_bit_cast(bf16x8_t, w);
}
__device__ __forceinline__ bf16x8_t seen_ones(uint32_t lo4, uint32_t hi4) {   // elements 0..3, 4..7 by bits 0..3 of each
  u32x4_t w;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t two = (j < 2 ? lo4 : hi4) >> (2 * (j & 1));
    w[j] = (two & 1 ? 0x3f80u : 0u) | (two & 2 ? 0x3f800000u : 0u);
  }
  return __builtin_bit_cast(bf16x8_t, w);
}
__device__ __forceinline__ void zero_not_finite(uint8_t* piece) {   // 16 bytes in LDS
  uint16_t* e = reinterpret_cast<uint16_t*>(piece);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if ((e[j] & 0x7f80u) == 0x7f80u) e[j] = 0;
}

// This workgroup's place among tiles of their own: 8 neighbours, which read much
// the same rows, to each of the 8 XCDs in turn (all of an XCD's in one piece
// would leave a prompt's long tiles to one of them). Two chunks of 2048 rows,
// window 512: 119.3 us in the order of the grid, 118.1 with this.
__device__ __forceinline__ int tile_wg() {
  constexpr unsigned kNear = 8;
  const unsigned id = blockIdx.x, whole = gridDim.x / (8 * kNear) * (8 * kNear), at = id >> 3;
  return (int)(id < whole ? at / kNear * (8 * kNear) + (id & 7) * kNear + at % kNear : id);
}

constexpr int kOutPitch = 272;               // bytes of a query's 128 output columns in LDS (256 + 16: bank spread)

// `n` queries' 128 columns (those below `most`) from LDS to their rows of the
// output, 16 lanes a query.
__device__ __forceinline__ void store_columns(uint16_t* out, const uint8_t* t, int most, int n, int lane) {
  for (int q0 = 0; q0 < n; q0 += 4) {
    const int mm = q0 + (lane >> 4);
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(t + mm * kOutPitch + (lane & 15) * 16);
    if (mm < most) *reinterpret_cast<u32x4_t*>(out + (int64_t)mm * kPagedVal + (lane & 15) * 8) = v;
  }
}

// A span's unnormalised output, in the order of the registers: 16 bytes per
// [workgroup][row tile][wave][column tile ct][j][lane] = columns 128 wave + 32
// ct + 8 j + 4 (lane / 32) .. +3 of query lane % 32 of the row tile, so that
// writing and joining move whole kilobytes.
__device__ __forceinline__ f32x4_t* part_at(float* part, int wg, int row_tiles, int r, int wave) {
  return reinterpret_cast<f32x4_t*>(part) + (((int64_t)wg * row_tiles + r) * 4 + wave) * 1024;
}
__device__ __forceinline__ void store_part(float* part, int wg, int row_tiles, const f32x16_t (&acc)[4][4], int wave,
                                           int lane) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (r < row_tiles) {
      f32x4_t* o = part_at(part, wg, row_tiles, r, wave) + lane;
#pragma unroll
      for (int ct = 0; ct < 4; ++ct)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[(ct * 4 + j) * 64] = f32x4_t{acc[ct][r][4 * j], acc[ct][r][4 * j + 1], acc[ct][r][4 * j + 2], acc[ct][r][4 * j + 3]};
    }
  }
}

// Workgroup = (tile of 128 queries of one sequence, span of its steps). With
// one span it writes out and lse; with several the span's maximum, sum and
// unnormalised output go to the workspace, and where its spans are to `info`.
//
// One wave per SIMD, so a step's phases overlap inside the wave: while the
// matrix cores form the scores of step i + 1, the vector unit turns those of
// step i into weights (the scheduler is told to put a few of its instructions
// behind each product); then a barrier, the value product of step i, and a
// barrier. Three step buffers: i (values), i + 1 (keys), i + 2 (loading, with
// a whole step's time to arrive). Rows arrive by direct-to-LDS loads: one
// instruction brings the 1024 bytes of a token's value part (the slot is
// scalar), one the last 128 bytes of eight tokens, in an order that spreads
// them over the banks. They are issued from inline asm, so that the compiler
// does not wait for them before every LDS read; they write no register, and a
// wave waits for all of its loads before the barrier that opens their step.
__global__ void __launch_bounds__(256, 1)
    paged_attn_kernel(const uint16_t* __restrict__ q, int64_t q_rs, int64_t q_hs, const uint8_t* __restrict__ pool, Pages pg,
                      const int32_t* __restrict__ row0, const int32_t* __restrict__ seq_len, int B, int T, int H,
                      int max_rows, int max_len, int window, int n_sink, float scale2, int planned, int row_tiles,
                      uint16_t* __restrict__ out, float* __restrict__ lse, float* __restrict__ part_o,
                      float2* __restrict__ part_ml, PartInfo* __restrict__ info) {
  __shared__ __align__(128) uint8_t tiles[kBufs * kTileB];
  __shared__ __align__(16) uint8_t ps[kMT * kPPitch];
  __shared__ float s_alpha[kMT], s_l[kMT];
  __shared__ int s_flag[4];   // per row tile: 1 = its maximum grew, 2 = a score that does not count is not finite

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, col = lane & 31, g = lane >> 5;
  const int wg = plan_wg();                                // in a plan
  Work wk;
  if (planned) {
    wk = plan_work<kMT, kStepTok>(row0, seq_len, pg, B, T, H, max_rows, max_len, window, n_sink, wg);
  } else {
    // more tiles than CUs: a tile each, the last (and in a chunk longest) first
    wk = tile_work(row0, seq_len, pg, B, T, H, max_rows, max_len, kMT, (int)gridDim.x - 1 - tile_wg());
  }
  const int b = wk.b, mt = wk.mt, sp = wk.sp, nsp = wk.n_span;
  const SeqRows sr = wk.sr;
  const int M = sr.n * H;                                  // fits: T H < 2^30 (checked on the host)
  const int m0 = mt * kMT;
  const int64_t mg0 = (int64_t)sr.first * H + m0;          // first query among the batch's (row, head) pairs
  if (planned) note_tile(info, wk, wg, mg0, min(kMT, M - m0), planned);
  if (b < 0) return;
  const int r_lo = m0 / H, r_hi = (min(m0 + kMT, M) - 1) / H;
  const int p_lo = sr.pos0 + r_lo, p_hi = sr.pos0 + r_hi;
  const Ranges rg = ranges_of<kStepTok>(p_lo, p_hi, window, n_sink);
  const int per = (rg.steps + nsp - 1) / nsp;
  const int step0 = min(sp * per, rg.steps), nsteps = min(step0 + per, rg.steps) - step0;

  float2* const my_ml = part_ml + (int64_t)wg * kMT;
  if (nsteps <= 0) {
    // nothing to see (a table without pages for it, a span past the end)
    for (int x = threadIdx.x; x < kMT; x += 256) {
      if (nsp > 1) my_ml[x] = make_float2(-__builtin_inff(), -1.f);   // no output of this span's is written
      else if (lse && x < M - m0) lse[mg0 + x] = -__builtin_inff();
    }
    if (nsp == 1)
      for (int x = threadIdx.x; x < min(kMT, M - m0) * (kPagedVal / 8); x += 256)
        reinterpret_cast<uint4*>(out + mg0 * kPagedVal)[x] = make_uint4(0, 0, 0, 0);
    return;
  }

  // this lane's query of row tile `wave`
  const int m = m0 + wave * 32 + col;
  const int mr = min(m, M - 1) / H, mh = min(m, M - 1) - mr * H;   // past the end: the last one again, never written
  const int p_row = sr.pos0 + mr;
  const int32_t* trow = pg.table + (int64_t)b * pg.ld;

  // tokens of step i: [t0, t0 + count)
  auto step_tok = [&](int i, int* count) -> int {
    const int st = step0 + i;
    const int t0 = st < rg.s0 ? st * kStepTok : rg.w0 + (st - rg.s0) * kStepTok;
    *count = min(kStepTok, (st < rg.s0 ? rg.n0 : rg.w1) - t0);
    return t0;
  };
  // The page of the step's token `lane` (lanes past the count: its last one),
  // and the slot it makes once the load is in.
  auto fetch_page = [&](int i, int& off) -> int {
    int cnt;
    const int t = step_tok(i, &cnt) + min(lane, cnt - 1);
    const uint32_t idx = page_index(pg, t);
    off = t - (int)idx * pg.size;
    return trow[idx];
  };
  auto slot_at = [&](int i, int page, int off) -> int {
    int cnt;
    step_tok(i, &cnt);
    return lane < cnt ? slot_in(pg, page, off) : -1;
  };
  // This wave's eight tokens of a step: 8 wave .. +7. A token without a slot
  // brings slot 0's row, which no query weighs.
  const uint32_t lds0 = lds_addr(tiles);
  auto issue_row = [&](int slot, int buf, int j) {
    const int tok = wave * 8 + j;
    const int sl = max(__builtin_amdgcn_readlane(slot, tok), 0);
    const uint8_t* src = pool + (uint64_t)(uint32_t)sl * (kPagedRow * 2);
    lds_load_row(lds0 + static_cast<uint32_t>(buf * kTileB + tok * kVPitch), lane * 16, src);
  };
  auto issue_tails = [&](int slot, int buf) {
    const int k = lane >> 3, tok = wave * 8 + k;
    const int sl = max(__shfl(slot, tok, 64), 0);
    const uint8_t* src = pool + (uint64_t)(uint32_t)sl * (kPagedRow * 2) + kPagedVal * 2 + (((lane & 7) ^ k) * 16);
    lds_load_lanes(lds0 + static_cast<uint32_t>(buf * kTileB + kTailAt + wave * 1024), src);
  };
  auto issue = [&](int slot, int buf) {
    issue_tails(slot, buf);
#pragma unroll
    for (int j = 0; j < 8; ++j) issue_row(slot, buf, j);
  };
  // key fragment s of the token `col` of a buffer
  const uint32_t k_off = col * kVPitch + g * 16, k_tail = kTailAt + col * 128 + ((g ^ (col & 7)) * 16);
  auto kload = [&](const uint8_t* buf, int s) -> bf16x8_t {
    return ld_bf16x8(buf + (s < 32 ? k_off + s * 32 : k_tail ^ ((s - 32) * 32)));   // tail pieces 2 (s - 32) + g, xor-ed
  };
  bf16x8_t qf[kKs16];   // the query, loaded behind the first rows
  f32x16_t acc[4][4];   // [column tile][row tile]
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[c][r][v] = 0.f;
  float mx = -__builtin_inff(), l = 0.f;   // running maximum of the query, this lane's part of its sum

  const uint8_t* const vlane = tiles + (4 * g + ((lane & 15) >> 2)) * kVPitch + wave * 256 + ((lane >> 4) & 1) * 32 + 8 * (lane & 3);
  // value fragment (V^T) of token half c, column tile ct: the contraction order
  // of a lane's 16 scores, tokens {16 c + 4 g .. +3, 16 c + 8 + 4 g .. +3}
  auto vload = [&](int buf, int c, int ct) -> bf16x8_t {
    const uint8_t* v = vlane + buf * kTileB + 16 * c * kVPitch + ct * 64;
    return ld_tr8(v, v + 8 * kVPitch);
  };
  uint8_t* const pmine = ps + (wave * 32 + col) * kPPitch + g * 16;
  const uint8_t* const pall = ps + col * kPPitch + g * 16;

  // The weights of a step from its scores st (lane: query col, tokens t0 + 8 (v
  // / 4) + 4 g + v % 4), a few instructions behind each of the first products
  // of the next step's scores nx. The order is the one written: a group per
  // product, closed by a scheduling barrier, key fragments kKD products ahead.
  bf16x8_t kb[kKD];
  auto weigh = [&](auto whole, f32x16_t& st, f32x16_t& nx, const uint8_t* kbuf, uint32_t bits) {
    constexpr bool FULL = decltype(whole)::value;
#pragma unroll
    for (int v = 0; v < 16; ++v) nx[v] = 0.f;
    float tmax = -__builtin_inff(), ref = 0.f, alpha = 1.f, psum = 0.f;
    bool poison = false, grow = false;
    bf16x8_t pb[2];
#pragma unroll
    for (int s = 0; s < kSplit; ++s) {
      nx = mfma32(kb[s % kKD], qf[s], nx);
      kb[s % kKD] = kload(kbuf, s + kKD);
      if (s < 8) {
#pragma unroll
        for (int v = 2 * s; v < 2 * s + 2; ++v) {
          float x = st[v] * scale2;
          if constexpr (!FULL) {
            const bool ok = (bits >> (8 * (v >> 2) + (v & 3))) & 1;
            poison |= !ok && !(fabsf(x) < __builtin_inff());
            x = ok ? x : -__builtin_inff();
          }
          st[v] = x;
          tmax = fmaxf(tmax, x);
        }
      } else if (s == 8) {
        tmax = pair_max(tmax);
      } else if (s == 9) {
        // the maximum moves only when a step's exceeds it by more than 8: a
        // weight may reach 2^8, and bf16 and fp32 keep their relative precision
        grow = __any(tmax > mx + 8.f);
        const float mn = grow ? fmaxf(mx, tmax) : mx;
        ref = mn == -__builtin_inff() ? 0.f : mn;
        alpha = grow ? __builtin_amdgcn_exp2f(mx - ref) : 1.f;   // 0 while nothing was seen
        mx = mn;
      } else if (s < 26) {
        const int v = s - 10;
        const float p = __builtin_amdgcn_exp2f(st[v] - ref);
        psum += p;
        pb[v >> 3][v & 7] = (__bf16)p;
        if (v == 7) *reinterpret_cast<u32x4_t*>(pmine) = __builtin_bit_cast(u32x4_t, pb[0]);
        if (v == 15) *reinterpret_cast<u32x4_t*>(pmine + 32) = __builtin_bit_cast(u32x4_t, pb[1]);
      } else if (s == 26) {
        l = l * alpha + psum;
        s_alpha[wave * 32 + col] = alpha;
        int flag = grow ? 1 : 0;
        if constexpr (!FULL) flag |= __any(poison) ? 2 : 0;
        s_flag[wave] = flag;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // the tokens of a step that this lane's query sees, as bits for its 16 scores
  auto seen_bits = [&](int t0, uint32_t ok) -> uint32_t {
    return (sees_bits(p_row, t0, window, n_sink) & ok) >> (4 * g);
  };
  auto whole_step = [&](int t0, uint32_t ok) -> bool {
    return ok == 0xffffffffu && t0 + kStepTok - 1 <= p_lo &&
           (window == 0 || t0 > p_hi - window || t0 + kStepTok <= n_sink);
  };
  // what the weights of a step change before its value product: accumulators of
  // grown maxima (none in the first step, they are 0), values that are not
  // finite; true if values changed
  auto adjust = [&](int cur, bool first, int t0, uint32_t ok) -> bool {
    int flags[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) flags[r] = __builtin_amdgcn_readfirstlane(s_flag[r]);
    const int any = flags[0] | flags[1] | flags[2] | flags[3];
    if (any == 0) return false;
    mfma32_acc_done();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if ((flags[r] & 1) && !first) {
        const float a = s_alpha[r * 32 + col];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          asm volatile("" : "+a"(acc[c][r]));   // one accumulator at a time leaves its registers
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[c][r][v] *= a;
          asm volatile("" : "+a"(acc[c][r]));
        }
      }
    }
    asm volatile("s_nop 7");
    if (!(any & 2)) return false;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int p = sr.pos0 + min(m0 + r * 32 + col, M - 1) / H;
      const uint32_t seen = (sees_bits(p, t0, window, n_sink) & ok) >> (4 * g);
      const bf16x8_t one0 = seen_ones(seen & 15u, (seen >> 8) & 15u), one1 = seen_ones((seen >> 16) & 15u, (seen >> 24) & 15u);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        f32x16_t n;
#pragma unroll
        for (int v = 0; v < 16; ++v) n[v] = 0.f;
        n = mfma32(not_finite(vload(cur, 0, c)), one0, n);
        n = mfma32(not_finite(vload(cur, 1, c)), one1, n);
        asm volatile("" : "+a"(acc[c][r]));
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[c][r][v] = n[v] != 0.f ? __builtin_nanf("") : acc[c][r][v];
        asm volatile("" : "+a"(acc[c][r]));
      }
    }
    asm volatile("s_nop 7");
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    for (int x = lane; x < kStepTok * 16; x += 64)   // in this wave's columns
      zero_not_finite(tiles + cur * kTileB + (x >> 4) * kVPitch + wave * 256 + (x & 15) * 16);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    return true;
  };
  auto pload = [&](int c, int r) -> bf16x8_t { return ld_bf16x8(pall + r * 32 * kPPitch + c * 32); };

  int page, off;                   // of the step to load next
  int slot2;                       // of step 2
  uint32_t ok0, ok1, ok2;          // tokens with a slot of steps i, i + 1, i + 2
  {
    // a span shorter than three steps loads its last one again
    int off0, off1, off2;
    const int i1 = min(1, nsteps - 1), i2 = min(2, nsteps - 1);
    const int page0 = fetch_page(0, off0), page1 = fetch_page(i1, off1), page2 = fetch_page(i2, off2);
    page = fetch_page(min(3, nsteps - 1), off);
    const int s0 = slot_at(0, page0, off0), s1 = slot_at(i1, page1, off1), s2 = slot_at(i2, page2, off2);
    ok0 = (uint32_t)__ballot(s0 >= 0);
    ok1 = (uint32_t)__ballot(s1 >= 0);
    ok2 = (uint32_t)__ballot(s2 >= 0);
    issue(s0, 0);
    issue(s1, 1);
    slot2 = s2;
  }
  {
    const uint8_t* qp = reinterpret_cast<const uint8_t*>(q + (int64_t)(sr.first + mr) * q_rs + (int64_t)mh * q_hs) + g * 16;
#pragma unroll
    for (int s = 0; s < kKs16; ++s) qf[s] = ld_bf16x8(qp + s * 32);
  }
  __builtin_amdgcn_s_waitcnt(0x70 | 0xF00);   // vmcnt(0): this wave's loads have landed
  __syncthreads();
  issue(slot2, 2);                 // read a round later: the queries do not wait for it
  f32x16_t st, nx;
#pragma unroll
  for (int v = 0; v < 16; ++v) st[v] = 0.f;
#pragma unroll
  for (int s = 0; s < kKD; ++s) kb[s] = kload(tiles, s);
#pragma unroll
  for (int s = 0; s < kKs16; ++s) {
    st = mfma32(kb[s % kKD], qf[s], st);
    kb[s % kKD] = s + kKD < kKs16 ? kload(tiles, s + kKD) : kload(tiles + kTileB, s + kKD - kKs16);
    __builtin_amdgcn_sched_barrier(0);
  }

  // Every round forms the scores of the next step and loads the one three
  // ahead; past the span's end these are repeats that nothing uses, which
  // keeps the round one straight piece of code.
  int cur = 0, nxt = 1, far = 2;   // buffers of steps i, i + 1, i + 2
  int cnt, t0 = step_tok(0, &cnt);
  auto round = [&](int i, f32x16_t& st, f32x16_t& nx) {
    // scores of step i + 1 beside the weights of step i
    const uint8_t* kbuf = tiles + nxt * kTileB;
    if (whole_step(t0, ok0)) weigh(std::true_type{}, st, nx, kbuf, 0);
    else weigh(std::false_type{}, st, nx, kbuf, seen_bits(t0, ok0));
    bf16x8_t vf[2], pf[2][4];
    vf[0] = vload(cur, 0, 0);
    vf[1] = vload(cur, 0, 1);
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
    // P and the flags cross while the last of those products run
#pragma unroll
    for (int r = 0; r < 4; ++r) pf[0][r] = pload(0, r);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = kSplit; s < kKs16; ++s) {
      nx = mfma32(kb[s % kKD], qf[s], nx);
      if (s + kKD < kKs16) kb[s % kKD] = kload(kbuf, s + kKD);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (adjust(cur, i == 0, t0, ok0)) {
      vf[0] = vload(cur, 0, 0);
      vf[1] = vload(cur, 0, 1);
    }
    __builtin_amdgcn_sched_barrier(0);
    // O^T += V^T P^T: a group per value fragment, two fragments ahead
#pragma unroll
    for (int x = 0; x < 6; ++x) {
      const int c = x >> 2, ct = x & 3;
#pragma unroll
      for (int r = 0; r < 4; ++r) mfma32_acc(acc[ct][r], vf[x & 1], pf[c][r]);
      vf[x & 1] = vload(cur, (x + 2) >> 2, (x + 2) & 3);
      if (x < 2) {
        pf[1][2 * x] = pload(1, 2 * x);
        pf[1][2 * x + 1] = pload(1, 2 * x + 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    const int slot = i + 3 < nsteps ? slot_at(i + 3, page, off) : -1;
    // Every wave has read its values and weights of step i, and its loads of
    // step i + 2 have landed.
    __builtin_amdgcn_s_waitcnt(0x70);           // vmcnt(0), lgkmcnt(0)
    __syncthreads();
    const uint8_t* kfar = tiles + far * kTileB;
    issue_tails(slot, cur);
#pragma unroll
    for (int x = 6; x < 8; ++x) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        mfma32_acc(acc[x & 3][r], vf[x & 1], pf[1][r]);
        if (x == 6 && r < kKD) kb[r] = kload(kfar, r);
        issue_row(slot, cur, (x - 6) * 4 + r);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    page = fetch_page(min(i + 4, nsteps - 1), off);   // in by the end of the next step
    ok0 = ok1;
    ok1 = ok2;
    ok2 = (uint32_t)__ballot(slot >= 0);
    t0 = step_tok(min(i + 1, nsteps - 1), &cnt);
    const int t = cur;
    cur = nxt;
    nxt = far;
    far = t;
  };
  for (int i = 0; i < nsteps; i += 2) {   // two at a time: the scores change places without a copy
    round(i, st, nx);
    if (i + 1 >= nsteps) break;
    round(i + 1, nx, st);
  }
  __builtin_amdgcn_s_waitcnt(0x70 | 0xF00);   // no load of a repeat is under way when the workgroup ends
  mfma32_acc_done();

  l = pair_sum(l);
  int tid = threadIdx.x;             // recomputed: held across the loop these would take registers it needs
  asm volatile("" : "+v"(tid));
  const int ecol = tid & 31, eg = (tid >> 5) & 1, elane = tid & 63;
  if (eg == 0) s_l[wave * 32 + ecol] = l;
  if (nsp > 1) {
    if (eg == 0) my_ml[wave * 32 + ecol] = make_float2(mx, l);
    store_part(part_o, wg, row_tiles, acc, wave, elane);
    return;
  }
  __syncthreads();                   // every wave's sums; and every wave is done with the step buffers
  if (lse && eg == 0 && m0 + wave * 32 + ecol < M)
    lse[mg0 + wave * 32 + ecol] = l == 0.f ? -__builtin_inff() : (mx + log2f(l)) * 0.69314718055994531f;
  // two row tiles at a time through this wave's part of the buffers, so that a
  // query's 128 columns leave as 256 bytes
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint8_t* const t = tiles + wave * (64 * kOutPitch);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = half * 2 + u;
      const float sl = s_l[r * 32 + ecol];
      const float inv = sl == 0.f ? 0.f : 1.f / sl;
#pragma unroll
      for (int ct = 0; ct < 4; ++ct)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bf16x4_t x;
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = (__bf16)(acc[ct][r][4 * j + e] * inv);
          *reinterpret_cast<uint2*>(t + (u * 32 + ecol) * kOutPitch + ct * 64 + j * 16 + eg * 8) = __builtin_bit_cast(uint2, x);
        }
    }
    store_columns(out + (mg0 + half * 64) * kPagedVal + wave * 128, t, M - m0 - half * 64, 64, elane);
  }
}

// ------------------------------------------------------------------ few queries
// The same for sequences of at most 32 queries (a decoded token of up to 32
// heads, two of 16): bound by the rows it reads, or, over short ranges, by the
// chain of waits of a round. A round takes 64 tokens. Wave w loads tokens 16 w
// .. +15 and forms their scores with all QT x 16 queries,
//   S^T[token][m] = K . Q^T       v_mfma_f32_16x16x32_bf16
// (four tokens of QT queries in a lane); the waves' maxima cross through LDS,
// the weights (4 KiB, after two lane swaps already the operand of the next
// product) cross too, and wave w adds value columns 128 w .. +127 of all 64:
//   O^T[col][m] += V^T . P^T      v_mfma_f32_32x32x16_bf16, 64 accumulators
// Two barriers a round; the next round's rows are asked for behind the first,
// when every wave has left the buffer they go to. Waves that are token lanes
// of their own, joined through LDS at the end, need no barrier but took 8.5K
// cycles to join: 64 sequences, one token, 32 heads, window 1024 of 100K 35 us,
// one token of 16 heads over 1000 19 us; with this 32 and 14 us.
constexpr int kNM = 32;                      // queries per workgroup
constexpr int kNTok = 16;                    // tokens per wave and round
constexpr int kNRound = 4 * kNTok;
constexpr int kNTail = kNRound * kVPitch;
constexpr int kNTile = kNTail + kNRound * 128;
constexpr int kNKs = kPagedRow / 32;         // contraction steps of the scores (18)
constexpr int kNKD = 6;                      // key fragments in flight

__device__ __forceinline__ f32x4_t mfma16(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  typedef __attribute__((__vector_size__(4 * sizeof(float)))) float v4_t;
  return __builtin_bit_cast(f32x4_t, __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, __builtin_bit_cast(v4_t, c), 0, 0, 0));
}
__device__ __forceinline__ float quad_max(float x) {   // over lanes l, l ^ 16, l ^ 32, l ^ 48
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return pair_max(fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1])));
}
__device__ __forceinline__ float quad_sum(float x) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return pair_sum(__uint_as_float(p[0]) + __uint_as_float(p[1]));
}

template <int QT>
__global__ void __launch_bounds__(256, 1)
    paged_attn_narrow_kernel(const uint16_t* __restrict__ q, int64_t q_rs, int64_t q_hs, const uint8_t* __restrict__ pool,
                             Pages pg, const int32_t* __restrict__ row0, const int32_t* __restrict__ seq_len, int B,
                             int T, int H, int max_rows, int max_len, int window, int n_sink, float scale2, int planned,
                             int row_tiles, uint16_t* __restrict__ out, float* __restrict__ lse,
                             float* __restrict__ part_o, float2* __restrict__ part_ml, PartInfo* __restrict__ info) {
  __shared__ __align__(128) uint8_t tiles[2 * kNTile];
  __shared__ __align__(16) uint8_t s_p[4 * 1024];   // P: per wave's tokens, a lane's 16 bytes
  __shared__ int s_page[4][2][64];   // per wave: page-table entries of two rounds' tokens
  __shared__ float s_x[4][kNM];      // per wave: a round's maximum of each query; at the end its sum
  __shared__ int s_poison[2][4];     // per wave: its tokens with a slot, and whether (bit 16) a score that does not count
                                     // is not finite; by the round's parity: a wave may write the next round's while
                                     // another reads

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, c16 = lane & 15, grp = lane >> 4, col = lane & 31, g = lane >> 5;
  const bool hi = (lane & 16) != 0;                        // query `col` is one of the second sixteen
  const int wg = plan_wg();                                // in a plan
  Work wk;
  if (planned) wk = plan_work<kNM, kNRound>(row0, seq_len, pg, B, T, H, max_rows, max_len, window, n_sink, wg);
  else wk = tile_work(row0, seq_len, pg, B, T, H, max_rows, max_len, kNM, (int)blockIdx.x);
  const int b = wk.b, sp = wk.sp, nsp = wk.n_span;
  const SeqRows sr = wk.sr;
  const int M = sr.n * H;                                  // 1 .. 16 QT
  const int64_t mg0 = (int64_t)sr.first * H;
  if (planned) note_tile(info, wk, wg, mg0, M, planned);
  if (b < 0) return;
  const Ranges rg = ranges_of<kNRound>(sr.pos0, sr.pos0 + sr.n - 1, window, n_sink);
  const int per = (rg.steps + nsp - 1) / nsp;
  const int round0 = min(sp * per, rg.steps), rounds = min(round0 + per, rg.steps) - round0;

  // tokens of this wave in round i: [t0, t0 + count), count <= 0: none
  auto round_tok = [&](int i, int* count) -> int {
    const int st = round0 + i;
    const int t0 = (st < rg.s0 ? st * kNRound : rg.w0 + (st - rg.s0) * kNRound) + wave * kNTok;
    *count = min(kNTok, (st < rg.s0 ? rg.n0 : rg.w1) - t0);
    return t0;
  };
  const int32_t* trow = pg.table + (int64_t)b * pg.ld;
  // entry and slot of the round's token c16 (past the count: its last, or token 0's)
  auto entry_of = [&](int i, int& off) -> const int32_t* {
    int cnt;
    const int t0 = round_tok(i, &cnt);
    const int t = cnt > 0 ? t0 + min(c16, cnt - 1) : 0;
    const uint32_t idx = page_index(pg, t);
    off = t - (int)idx * pg.size;
    return trow + idx;
  };
  auto slot_at = [&](int i, int page, int off) -> int {
    int cnt;
    round_tok(i, &cnt);
    const int sl = slot_in(pg, page, off);
    return c16 < cnt ? sl : -1;
  };
  const uint32_t lds0 = lds_addr(tiles), page0 = lds_addr(&s_page[wave][0][0]);
  auto issue_pages = [&](int i) {
    int off;
    lds_load_dwords(page0 + (i & 1) * 256u, entry_of(min(i, rounds - 1), off));
  };
  // a token without a slot brings slot 0's row, which no query weighs
  auto issue = [&](int slot, int buf) {
    const uint32_t base = lds0 + static_cast<uint32_t>(buf * kNTile + wave * kNTok * kVPitch);
    const uint32_t tail = lds0 + static_cast<uint32_t>(buf * kNTile + kNTail + wave * kNTok * 128);
#pragma unroll
    for (int j = 0; j < kNTok; ++j) {
      const int sl = max(__builtin_amdgcn_readlane(slot, j), 0);
      lds_load_row(base + j * kVPitch, lane * 16, pool + (uint64_t)(uint32_t)sl * (kPagedRow * 2));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = lane >> 3, sl = max(__shfl(slot, j * 8 + k, 64), 0);
      lds_load_lanes(tail + j * 1024, pool + (uint64_t)(uint32_t)sl * (kPagedRow * 2) + kPagedVal * 2 + (((lane & 7) ^ k) * 16));
    }
  };
  // key fragment s (32 values) of this wave's token c16: its piece 4 s + grp
  const uint32_t k_off = (wave * kNTok + c16) * kVPitch + grp * 16, k_tail = kNTail + (wave * kNTok + c16) * 128;
  auto kload = [&](const uint8_t* buf, int s) -> bf16x8_t {
    return ld_bf16x8(buf + (s < 16 ? k_off + s * 64 : k_tail + (((4 * (s - 16) + grp) ^ (c16 & 7)) * 16)));
  };
  // value fragment (V^T) of this wave's column tile ct, tokens 16 kk + 8 g .. +7
  const uint32_t v_off = (8 * g + (c16 >> 2)) * kVPitch + wave * 256 + ((lane >> 4) & 1) * 32 + 8 * (lane & 3);
  auto vload = [&](const uint8_t* buf, int kk, int ct) -> bf16x8_t {
    const uint8_t* v = buf + v_off + kk * 16 * kVPitch + ct * 64;
    return ld_tr8(v, v + 4 * kVPitch);
  };

  f32x16_t acc[4];    // [column tile]: O^T[col][query col]
  float mx[QT], l[QT];   // of queries c16, 16 + c16: the same in every wave; this lane's part of this wave's
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[c][v] = 0.f;
#pragma unroll
  for (int h = 0; h < QT; ++h) {
    mx[h] = -__builtin_inff();
    l[h] = 0.f;
  }

  if (rounds > 0) {
    int p_row[QT];
    bf16x8_t qf[QT][kNKs];
    int slot;
    {
      int off0;
      const int page = *entry_of(0, off0);
      slot = slot_at(0, page, off0);
      issue_pages(1);
      issue(slot, 0);
    }
#pragma unroll
    for (int h = 0; h < QT; ++h) {
      const int m = min(16 * h + c16, M - 1), mr = m / H, mh = m - mr * H;   // past the end: the last one again
      p_row[h] = sr.pos0 + mr;
      const uint8_t* qp = reinterpret_cast<const uint8_t*>(q + (int64_t)(sr.first + mr) * q_rs + (int64_t)mh * q_hs) + grp * 16;
#pragma unroll
      for (int s = 0; s < kNKs; ++s) qf[h][s] = ld_bf16x8(qp + s * 64);
    }
    for (int i = 0; i < rounds; ++i) {
      __builtin_amdgcn_s_waitcnt(0x70 | 0xF00);   // vmcnt(0): this wave's rows of round i, the entries of round i + 1
      asm volatile("" ::: "memory");
      const uint8_t* buf = tiles + (i & 1) * kNTile;
      int cnt;
      const int t0 = round_tok(i, &cnt);
      const uint32_t ok = (uint32_t)__ballot(slot >= 0) & 0xffffu;
      f32x4_t st[QT];
#pragma unroll
      for (int h = 0; h < QT; ++h) st[h] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      bf16x8_t kb[kNKD];
#pragma unroll
      for (int s = 0; s < kNKD; ++s) kb[s] = kload(buf, s);
#pragma unroll
      for (int s = 0; s < kNKs; ++s) {
#pragma unroll
        for (int h = 0; h < QT; ++h) st[h] = mfma16(kb[s % kNKD], qf[h][s], st[h]);
        if (s + kNKD < kNKs) kb[s % kNKD] = kload(buf, s + kNKD);
        __builtin_amdgcn_sched_barrier(0);
      }
      float tmax[QT];
      bool poison = false;   // a score that does not count is not finite: its row holds infinities or NaN
      {
        const bool whole = ok == 0xffffu && t0 + kNTok - 1 <= sr.pos0 &&
                           (window == 0 || t0 > sr.pos0 + sr.n - 1 - window || t0 + kNTok <= n_sink);
#pragma unroll
        for (int h = 0; h < QT; ++h) {
          const uint32_t bits = whole ? 0xffffu : (sees_bits(p_row[h], t0, window, n_sink) & ok);
          tmax[h] = -__builtin_inff();
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float x = st[h][v] * scale2;
            const bool seen = (bits >> (4 * grp + v)) & 1;
            poison |= !seen && !(fabsf(x) < __builtin_inff());
            st[h][v] = seen ? x : -__builtin_inff();
            tmax[h] = fmaxf(tmax[h], st[h][v]);
          }
          tmax[h] = quad_max(tmax[h]);
        }
      }
      s_x[wave][col] = QT == 2 && hi ? tmax[QT - 1] : tmax[0];   // lanes l and l ^ 32 write the same
      s_poison[i & 1][wave] = (int)ok | (__any(poison) ? 0x10000 : 0);
      __syncthreads();
      // every wave has left round i - 1: its buffer takes round i + 1
      int next = -1;
      if (i + 1 < rounds) {
        int off;
        entry_of(i + 1, off);
        next = slot_at(i + 1, s_page[wave][(i + 1) & 1][lane], off);
        issue_pages(i + 2);
        issue(next, (i + 1) & 1);
      }
      float alpha[QT];
      uint32_t pk[2][2] = {{0u, 0u}, {0u, 0u}};
      bool grown = false;
#pragma unroll
      for (int h = 0; h < QT; ++h) {
        float top = s_x[0][16 * h + c16];
#pragma unroll
        for (int w = 1; w < 4; ++w) top = fmaxf(top, s_x[w][16 * h + c16]);
        const bool grow = __any(top > mx[h] + 8.f);            // as in the 128-query kernel; alike in every wave
        const float mn = grow ? fmaxf(mx[h], top) : mx[h];
        const float ref = mn == -__builtin_inff() ? 0.f : mn;
        alpha[h] = grow ? __builtin_amdgcn_exp2f(mx[h] - ref) : 1.f;
        grown |= grow;
        float p[4], psum = 0.f;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          p[v] = __builtin_amdgcn_exp2f(st[h][v] - ref);
          psum += p[v];
        }
        const bf16x4_t pb = {(__bf16)p[0], (__bf16)p[1], (__bf16)p[2], (__bf16)p[3]};
        const uint2 u = __builtin_bit_cast(uint2, pb);
        pk[h][0] = u.x;
        pk[h][1] = u.y;
        l[h] = l[h] * alpha[h] + psum;
        mx[h] = mn;
      }
      // Lane group r holds tokens 4 r .. +3 of queries c16 and 16 + c16; after
      // the swaps lane l holds tokens 8 g .. +7 of query l % 32.
      {
        const auto s01 = __builtin_amdgcn_permlane16_swap(pk[0][0], pk[1][0], false, false);
        const auto s23 = __builtin_amdgcn_permlane16_swap(pk[0][1], pk[1][1], false, false);
        *reinterpret_cast<u32x4_t*>(s_p + wave * 1024 + lane * 16) = u32x4_t{s01[0], s23[0], s01[1], s23[1]};
      }
      if (grown && i > 0) {
        const float a = QT == 2 && hi ? alpha[QT - 1] : alpha[0];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[c][v] *= a;
      }
      __syncthreads();                            // P, and every wave's rows, are there
      const int* const bad = s_poison[i & 1];
      if ((bad[0] | bad[1] | bad[2] | bad[3]) & 0x10000) {
        // as in the 128-query kernel, each wave in its columns
        const int p = sr.pos0 + min(col, M - 1) / H;
#pragma unroll 1   // rare: nothing of it is kept in registers across rounds
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t seen = (sees_bits(p, t0 + (kk - wave) * kNTok, window, n_sink) & (uint32_t)bad[kk] & 0xffffu) >> (8 * g);
          const bf16x8_t ones = seen_ones(seen & 15u, (seen >> 4) & 15u);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            f32x16_t n;
#pragma unroll
            for (int v = 0; v < 16; ++v) n[v] = 0.f;
            n = mfma32(not_finite(vload(buf, kk, c)), ones, n);
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[c][v] = n[v] != 0.f ? __builtin_nanf("") : acc[c][v];
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        uint8_t* wbuf = tiles + (i & 1) * kNTile + wave * 256;
        for (int y = lane; y < kNRound * 16; y += 64) zero_not_finite(wbuf + (y >> 4) * kVPitch + (y & 15) * 16);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
      bf16x8_t pf[4], vf[4];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) pf[kk] = ld_bf16x8(s_p + kk * 1024 + lane * 16);
#pragma unroll
      for (int x = 0; x < 4; ++x) vf[x] = vload(buf, 0, x);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        acc[x & 3] = mfma32(vf[x & 3], pf[x >> 2], acc[x & 3]);
        if (x + 4 < 16) vf[x & 3] = vload(buf, (x + 4) >> 2, x & 3);
        __builtin_amdgcn_sched_barrier(0);
      }
      slot = next;
    }
  }

  // the waves' sums: query l % 32 of every lane
  __syncthreads();                                // s_x of the last round is read
  {
    float x = quad_sum(l[0]);
    if (QT == 2) {
      const float y = quad_sum(l[QT - 1]);
      x = hi ? y : x;
    }
    s_x[wave][col] = x;
  }
  __syncthreads();
  const float den = (s_x[0][col] + s_x[1][col]) + (s_x[2][col] + s_x[3][col]);
  const float top = QT == 2 && hi ? mx[QT - 1] : mx[0];
  if (nsp > 1) {
    if (wave == 0 && g == 0) part_ml[(int64_t)wg * kMT + col] = make_float2(top, den);
    f32x4_t* o = part_at(part_o, wg, row_tiles, 0, wave) + lane;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[(c * 4 + j) * 64] = f32x4_t{acc[c][4 * j], acc[c][4 * j + 1], acc[c][4 * j + 2], acc[c][4 * j + 3]};
    return;
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  if (lse && wave == 0 && g == 0 && col < M)
    lse[mg0 + col] = den == 0.f ? -__builtin_inff() : (top + log2f(den)) * 0.69314718055994531f;
  uint8_t* const t = tiles + wave * (32 * kOutPitch);   // every wave has left the buffers
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf16x4_t x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = (__bf16)(acc[c][4 * j + e] * inv);
      *reinterpret_cast<uint2*>(t + col * kOutPitch + c * 64 + j * 16 + g * 8) = __builtin_bit_cast(uint2, x);
    }
  store_columns(out + mg0 * kPagedVal + wave * 128, t, M, 32, lane);
}

// out and lse of the tiles that took several spans, in span order. grid (tiles,
// 16 x row tiles), 256 threads: a workgroup joins 32 columns of 32 queries, a
// thread one 16-byte piece, kG spans' loads under way at a time.
constexpr int kG = 8;
constexpr int kJoinPitch = 80;               // bytes of a query's 32 columns in LDS (64 + 16: bank spread)
__global__ void __launch_bounds__(256)
    paged_attn_merge_kernel(const float* __restrict__ part_o, const float2* __restrict__ part_ml,
                            const PartInfo* __restrict__ info, int row_tiles, uint16_t* __restrict__ out,
                            float* __restrict__ lse) {
  __shared__ __align__(16) uint8_t t[32 * kJoinPitch];
  const int r = blockIdx.y >> 4, cw = (blockIdx.y >> 2) & 3, ct = blockIdx.y & 3;
  const PartInfo in = info[blockIdx.x];
  const int n = in.n_span, most = in.queries - r * 32;
  if (n <= 1 || most <= 0 || in.base < 0 || in.base > kCus - n) return;   // one span wrote its output itself
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 31, g = lane >> 5;
  const float2* ml = part_ml + (int64_t)in.base * kMT + r * 32 + col;
  const f32x4_t* po = part_at(const_cast<float*>(part_o), in.base, row_tiles, r, cw) + ct * 256 + threadIdx.x;
  const int64_t stride = (int64_t)row_tiles * 4 * 1024;
  float mx = -__builtin_inff(), den = 0.f;
  f32x4_t o = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < n; s0 += kG) {
    float2 a[kG];
    f32x4_t x[kG];
#pragma unroll
    for (int u = 0; u < kG; ++u) {
      a[u] = make_float2(-__builtin_inff(), -1.f);
      x[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (s0 + u < n) {                                     // uniform: no load is repeated, none waits
        a[u] = ml[(int64_t)(s0 + u) * kMT];
        x[u] = po[(s0 + u) * stride];
      }
    }
    float top = mx;
#pragma unroll
    for (int u = 0; u < kG; ++u) top = fmaxf(top, a[u].x);
    const float ref = top == -__builtin_inff() ? 0.f : top;
    const float f = exp2f((mx == -__builtin_inff() ? ref : mx) - ref);   // o and den are 0 before anything is seen
    den *= f;
    o *= f;
#pragma unroll
    for (int u = 0; u < kG; ++u) {
      if (!(a[u].y < 0.f)) {                  // below 0: a span without steps, which wrote no output
        const float w = exp2f((a[u].x == -__builtin_inff() ? ref : a[u].x) - ref);
        den += w * a[u].y;
        o += w * x[u];
      }
    }
    mx = top;
  }
  if (lse && cw == 0 && ct == 0 && wave == 0 && g == 0 && col < most)
    lse[in.first + r * 32 + col] = den == 0.f ? -__builtin_inff() : (mx + log2f(den)) * 0.69314718055994531f;
  const float inv = den == 0.f ? 0.f : 1.f / den;
  bf16x4_t y;                         // this thread's piece: columns 8 wave + 4 g .. +3 of query col
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = (__bf16)(o[e] * inv);
  *reinterpret_cast<uint2*>(t + col * kJoinPitch + wave * 16 + g * 8) = __builtin_bit_cast(uint2, y);
  __syncthreads();
  const int mm = threadIdx.x >> 2;    // 32 queries x 64 bytes, four threads a query
  if (mm < min(most, 32))
    *reinterpret_cast<u32x4_t*>(out + (in.first + r * 32 + mm) * kPagedVal + cw * 128 + ct * 32 + (threadIdx.x & 3) * 8) =
        *reinterpret_cast<const u32x4_t*>(t + mm * kJoinPitch + (threadIdx.x & 3) * 16);
}

// Upper bound of the batch's tiles, when no row is two sequences': every
// sequence rounds up once.
int64_t tiles_of(int B, int T, int H, int64_t per_seq, int per) {
  return std::min<int64_t>(B * per_seq, (int64_t)T * H / per + B);
}

// Whether tiles are split over spans, and what the workspace holds then. At most
// 32 queries a sequence take the narrow kernel (one token of 16 heads over 1000:
// 13.1 us, the wide one 18.3; 64 tokens of 32 heads, window 1024: 31.0, 36.4),
// at most 16 its form with one query a lane (13.1, with two 13.6). Up to 256
// tiles are split (32 tokens of 128 heads over 8K to 16K 151 us, not split 881;
// 12 chunks of 77 rows 71, 282; window 1024 31, 50); more fill the CUs unsplit.
struct Split {
  bool narrow;        // at most 32 queries a sequence
  bool planned;
  int64_t tiles;
  int row_tiles;      // of 32 queries a partial holds
  size_t part_o, part_ml, info, bytes;
};
Split split_of(int B, int T, int H, int max_rows, int max_len, int window, int n_sink) {
  Split sp{};
  sp.narrow = (int64_t)std::min(max_rows, T) * H <= kNM;
  const int per = sp.narrow ? kNM : kMT;
  const int64_t per_seq = ((int64_t)std::min(max_rows, T) * H + per - 1) / per;
  sp.tiles = tiles_of(B, T, H, per_seq, per);
  int64_t seen = max_len;                                  // tokens a tile can read
  if (window > 0) seen = std::min<int64_t>(seen, (int64_t)window + n_sink + kMT / H + 1 + kStepTok);
  sp.planned = sp.tiles <= kCus && seen > kMinSpan * kStepTok && plan_fits(B, B * per_seq, seen);
  if (!sp.planned) return sp;
  sp.row_tiles = (int)((std::min<int64_t>(per, (int64_t)std::min(max_rows, T) * H) + 31) / 32);
  sp.part_ml = (size_t)kCus * sp.row_tiles * 32 * kPagedVal * sizeof(float);
  sp.info = sp.part_ml + (size_t)kCus * kMT * sizeof(float2);
  sp.bytes = sp.info + (size_t)kCus * sizeof(PartInfo);
  return sp;
}

bool shape_ok(int B, int T, int H, int max_rows, int max_len, int window, int n_sink) {
  return batch_ok(B, T, max_rows, max_len) && H >= 1 && H <= 128 && (int64_t)T * H < (1ll << 30) && window >= 0 &&
         n_sink >= 0;
}

}  // namespace

extern "C" size_t ech_paged_attn_ws_bytes(int B, int T, int H, int max_rows, int max_len, int window, int n_sink) {
  if (!shape_ok(B, T, H, max_rows, max_len, window, n_sink) || T == 0 || max_rows == 0) return 0;
  return split_of(B, T, H, max_rows, max_len, window, n_sink).bytes;
}

extern "C" int ech_paged_attn(const void* q, int64_t q_row_stride, int64_t q_head_stride, const void* pool,
                              int64_t n_slots, int page_size, const int32_t* page_table, int64_t pt_ld,
                              const int32_t* row0, const int32_t* seq_len, int B, int T, int H, int max_rows,
                              int max_len, int window, int n_sink, float sm_scale, void* out, float* lse, void* ws,
                              size_t ws_bytes, void* stream) {
  if (!pool || !row0 || !seq_len || (T > 0 && (!q || !out))) return ECH_EINVAL;
  if (!shape_ok(B, T, H, max_rows, max_len, window, n_sink) || !pages_ok(n_slots, page_size, page_table, pt_ld))
    return ECH_EINVAL;
  if (!(sm_scale == sm_scale) || !aligned16_(q) || !aligned16_(pool) || !aligned16_(out) || q_row_stride < 0 ||
      q_head_stride < 0 || q_row_stride % 8 || q_head_stride % 8)
    return ECH_EINVAL;
  const size_t need = ech_paged_attn_ws_bytes(B, T, H, max_rows, max_len, window, n_sink);
  if (ws_bytes < need || (need && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u)))) return ECH_EINVAL;
  if (T == 0 || max_rows == 0) return ECH_OK;
  if (window >= max_len) window = 0;                       // no position has more tokens behind it
  n_sink = std::min(n_sink, max_len);
  const Split sp = split_of(B, T, H, max_rows, max_len, window, n_sink);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  char* w = static_cast<char*>(ws);
  float* part_o = reinterpret_cast<float*>(w);
  float2* part_ml = sp.planned ? reinterpret_cast<float2*>(w + sp.part_ml) : nullptr;
  PartInfo* info = sp.planned ? reinterpret_cast<PartInfo*>(w + sp.info) : nullptr;
  const Pages pg = make_pages(page_table, pt_ld, n_slots, page_size);
  const int64_t queries = (int64_t)std::min(max_rows, T) * H;
  const auto kernel = !sp.narrow ? paged_attn_kernel : queries <= 16 ? paged_attn_narrow_kernel<1> : paged_attn_narrow_kernel<2>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(sp.planned ? kCus : sp.tiles)), dim3(256), 0, s,
                     static_cast<const uint16_t*>(q), q_row_stride, q_head_stride, static_cast<const uint8_t*>(pool), pg,
                     row0, seq_len, B, T, H, max_rows, max_len, window, n_sink, sm_scale * 1.4426950408889634f,
                     sp.planned ? (int)sp.tiles : 0, sp.row_tiles, static_cast<uint16_t*>(out), lse, part_o, part_ml, info);
  ECH_LAUNCH_CHECK();
  if (sp.planned) {
    hipLaunchKernelGGL(paged_attn_merge_kernel, dim3((unsigned)sp.tiles, 16 * sp.row_tiles), dim3(256), 0, s, part_o, part_ml, info,
                       sp.row_tiles, static_cast<uint16_t*>(out), lse);
    ECH_LAUNCH_CHECK();
  }
  return ECH_OK;
}
