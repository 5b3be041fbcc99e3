// The attention weight that each cached token received (ech_paged_weight):
//
//   acc_out[b][t] = decay acc_in[b][t] + sum over the step's rows i of b that
//                   see t, and heads h, of exp(scale q[i][h] . k[t] - lse[i][h])
//
// with the lse of ech_paged_attn, so each (row, head) hands out exactly 1. Two
// forms, both S[m][token] = Q . K^T on v_mfma_f32_32x32x16_bf16, which leaves a
// lane one token and 16 queries, so that the sum over queries stays in the
// lane; the weights are formed a step late, between the products of the next
// step. No other lane or workgroup adds to a token out of order: the same call
// gives the same bits.
//  - Sequences of at most 128 queries (decoding): the queries stay in registers
//    and the rows stream past them; bound by the rows' bytes: 32 tokens of 128
//    heads over 8K to 16K tokens 104-109 us, 4.2 TB/s (the other form 164 us;
//    a whole sequence per workgroup 962 us).
//  - More queries (chunks), which this form would have to pass the rows by more
//    than once: 256 tokens' rows stay in registers (64 a wave, 288 registers)
//    and the queries stream past. 4 chunks of 64 rows at 64 heads over 10K tokens
//    213-218 us, 880 TF/s: 480 workgroups in two rounds on 256 CUs, each with 22K
//    cycles to start and 43 steps of 4300 (the products 2304), at 2.3 GHz while
//    the call runs over and over (1.9 in the first 20 calls, 250 us each). Those
//    of the last tokens look at the mask in every step and take 5350: two of them
//    in a row on a CU end the kernel at 210 us, the others end at 181. With the
//    row loads and the weights' instructions spread between the products a step
//    takes 3774 cycles, but 5290 with the mask and at 2.16 GHz: 215 us.
#include <algorithm>

#include "common.hpp"
#include "paged_tile.hpp"

namespace {

constexpr int kBufs = 3;
constexpr int kLoads = 9;                    // row loads of a wave per step
constexpr float kLog2e = 1.4426950408889634f;

// Fragment s (16 values) of row `col` of a step buffer: piece 2 s + g.
__device__ __forceinline__ bf16x8_t row_frag(const uint8_t* buf, int col, int g, int s) {
  return s < 32 ? ld_bf16x8(buf + col * kVPitch + g * 16 + s * 32)
                : ld_bf16x8(buf + kTailAt + col * 128 + (((2 * (s - 32) + g) ^ (col & 7)) * 16));
}

// ------------------------------------------------------------------ few queries
// Workgroup = a span of 32-token steps of one sequence; wave w holds queries 32
// w .. +31. Step buffers: i (read), i + 1 and i + 2 (under way). A step's sums
// go to LDS per wave and are joined and written kChunk steps at a time.
constexpr int kMS = 128;
constexpr int kChunk = 64;
__global__ void __launch_bounds__(256, 1)
    paged_weight_stream_kernel(const uint16_t* __restrict__ q, int64_t q_rs, int64_t q_hs, const float* __restrict__ lse,
                               const uint8_t* __restrict__ pool, Pages pg, const int32_t* __restrict__ row0,
                               const int32_t* __restrict__ seq_len, int B, int T, int H, int max_rows, int max_len,
                               int window, int n_sink, float scale2, int planned, const float* acc_in, float* acc_out,
                               int64_t acc_ld, float decay) {
  __shared__ __align__(128) uint8_t tiles[kBufs * kTileB];
  __shared__ float s_w[4][kChunk * kStepTok];
  __shared__ int s_page[4][2][64];   // per wave: page-table entries of two steps' tokens
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, col = lane & 31, g = lane >> 5;
  Work wk;
  if (planned) {
    if (window == 0)
      wk = plan_work<kMS, kStepTok, true>(row0, seq_len, pg, B, T, H, max_rows, max_len, window, n_sink, blockIdx.x);
    else
      wk = plan_work<kMS, kStepTok>(row0, seq_len, pg, B, T, H, max_rows, max_len, window, n_sink, blockIdx.x);
  } else {
    wk = Work{(int)blockIdx.x, 0, 0, 1, seq_rows(row0, seq_len, pg, blockIdx.x, T, max_rows, max_len), 0, 0};
  }
  const int b = __builtin_amdgcn_readfirstlane(wk.b);
  const int sp = __builtin_amdgcn_readfirstlane(wk.sp), nsp = __builtin_amdgcn_readfirstlane(wk.n_span);
  if (b < 0) return;
  const SeqRows sr = wk.sr;
  const int M = sr.n * H;
  // without a window all tokens are written here (the last ones by rows that see
  // them, those of a sequence without rows by nobody's weight); with one, those
  // that some row sees, the decay of the others being done before
  const Ranges rg = window == 0 ? ranges_of<kStepTok>(sr.len - 1, sr.len - 1, 0, 0)
                                : ranges_of<kStepTok>(sr.pos0, sr.pos0 + sr.n - 1, window, n_sink);
  if (window != 0 && M == 0) return;
  const int per = (rg.steps + nsp - 1) / nsp;
  const int step0 = min(sp * per, rg.steps), nsteps = min(step0 + per, rg.steps) - step0;
  if (nsteps <= 0) return;
  const float* in = acc_in ? acc_in + (int64_t)b * acc_ld : nullptr;
  float* to = acc_out + (int64_t)b * acc_ld;
  const int32_t* trow = pg.table + (int64_t)b * pg.ld;

  auto step_tok = [&](int i, int* count) -> int {
    const int st = step0 + i;
    const int t0 = st < rg.s0 ? st * kStepTok : rg.w0 + (st - rg.s0) * kStepTok;
    *count = min(kStepTok, (st < rg.s0 ? rg.n0 : rg.w1) - t0);
    return t0;
  };
  // steps [c0, c1) joined over the waves and written
  auto write_chunk = [&](int c0, int c1, bool weights) {
    for (int x = threadIdx.x; x < (c1 - c0) * kStepTok; x += 256) {
      int cnt;
      const int t0 = step_tok(c0 + x / kStepTok, &cnt), k = x % kStepTok;
      if (k < cnt) {
        const float w = weights ? (s_w[0][x] + s_w[1][x]) + (s_w[2][x] + s_w[3][x]) : 0.f;
        to[t0 + k] = (in ? in[t0 + k] * decay : 0.f) + w;
      }
    }
  };
  if (M == 0) {
    for (int c0 = 0; c0 < nsteps; c0 += kChunk) write_chunk(c0, min(c0 + kChunk, nsteps), false);
    return;
  }

  auto entry_of = [&](int i, int& off) -> const int32_t* {
    int cnt;
    const int t = step_tok(i, &cnt) + min(col, cnt - 1);
    const uint32_t idx = page_index(pg, t);
    off = t - (int)idx * pg.size;
    return trow + idx;
  };
  // slot of the step's token `col` (-1: none)
  auto slot_at = [&](int i, int page, int off) -> int {
    int cnt;
    step_tok(i, &cnt);
    const int sl = slot_in(pg, page, off);
    return col < cnt ? sl : -1;
  };
  const uint32_t lds0 = lds_addr(tiles), page0 = lds_addr(&s_page[wave][0][0]);
  auto issue_pages = [&](int i) {
    int off;
    lds_load_dwords(page0 + (i & 1) * 256u, entry_of(min(i, nsteps - 1), off));
  };
  auto issue = [&](int slot, int buf) {
    const uint32_t base = lds0 + static_cast<uint32_t>(buf * kTileB);
    const int k = lane >> 3;
    const int st = max(__shfl(slot, wave * 8 + k, 64), 0);
    lds_load_lanes(base + kTailAt + wave * 1024,
                   pool + (uint64_t)(uint32_t)st * (kPagedRow * 2) + kPagedVal * 2 + (((lane & 7) ^ k) * 16));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int sl = max(__builtin_amdgcn_readlane(slot, wave * 8 + j), 0);
      lds_load_row(base + (wave * 8 + j) * kVPitch, lane * 16, pool + (uint64_t)(uint32_t)sl * (kPagedRow * 2));
    }
  };

  int slot0, slot1, slot_t;                   // slots of steps i, i + 1 and of the step to load
  {
    int off0, off1;
    const int i1 = min(1, nsteps - 1);
    const int p0 = *entry_of(0, off0), p1 = *entry_of(i1, off1);
    slot0 = slot_at(0, p0, off0);
    slot1 = slot_at(i1, p1, off1);
  }
  issue(slot0, 0);
  bf16x8_t qf[kKs16];
  float ls[16];                               // lse of query 32 w + 8 (v / 4) + 4 g + v % 4, base 2
  int ps[16];                                 // its position; past the last query: sees nothing
  {
    const int m = min(wave * 32 + col, M - 1), mr = m / H, mh = m - mr * H;
    const uint8_t* qp = reinterpret_cast<const uint8_t*>(q + (int64_t)(sr.first + mr) * q_rs + (int64_t)mh * q_hs) + g * 16;
#pragma unroll
    for (int s = 0; s < kKs16; ++s) qf[s] = ld_bf16x8(qp + s * 32);
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int mv = wave * 32 + 8 * (v >> 2) + 4 * g + (v & 3), mc = min(mv, M - 1);
      ls[v] = lse[(int64_t)sr.first * H + mc] * kLog2e;
      ps[v] = mv < M ? sr.pos0 + mc / H : -1;
    }
  }
  __builtin_amdgcn_s_waitcnt(0x70 | 0xF00);   // vmcnt(0): step 0, the queries
  issue_pages(2);
  issue(slot1, 1);
  const bool active = wave * 32 < M;          // the wave has queries
  const bool even = wave * 32 + 32 <= M;      // and all 32 of them

  f32x16_t st, nx;
#pragma unroll
  for (int v = 0; v < 16; ++v) st[v] = 0.f;
  // The weights of the scores st of step j (its token's slot there or not) in
  // pieces: one query per call.
  float sum[2];
  const int win = window == 0 ? 0x40000000 : window;   // positions are below 2^30
  auto piece = [&](int v, bool whole, int t, bool there) {
    const float e = __builtin_amdgcn_exp2f(fmaf(st[v], scale2, -ls[v]));
    const bool seen = whole | (there & (t <= ps[v]) & ((t > ps[v] - win) | (t < n_sink)));
    sum[v & 1] += seen ? e : 0.f;
  };
  bool p_whole = false, p_there = false;
  int p_t = 0;
  for (int i = 0; i <= nsteps; ++i) {
    // step i has landed (all but the newest step's loads), step i - 1 is read
    if (i < nsteps) __builtin_amdgcn_s_waitcnt(0x70 | 0xF00 | kLoads);
    __syncthreads();
    if (i > 1 && (i - 1) % kChunk == 0) {
      // sums of steps up to i - 2 are in LDS
      write_chunk(i - 1 - kChunk, i - 1, true);
      __builtin_amdgcn_s_waitcnt(0x70 | 0xF00);
      __syncthreads();
    }
    const uint8_t* buf = tiles + (i % kBufs) * kTileB;
    if (i < nsteps) {
      int off;
      const int j = min(i + 2, nsteps - 1);
      entry_of(j, off);
      const int sl = slot_at(j, s_page[wave][i & 1][lane], off);
      slot_t = i + 2 < nsteps ? sl : -1;
      issue_pages(i + 3);
      issue(slot_t, (i + 2) % kBufs);
    }
    sum[0] = sum[1] = 0.f;
    if (active) {
      if (i < nsteps) {
        constexpr int kD = 5;
        bf16x8_t kb[kD];
#pragma unroll
        for (int v = 0; v < 16; ++v) nx[v] = 0.f;
#pragma unroll
        for (int s = 0; s < kD; ++s) kb[s] = row_frag(buf, col, g, s);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < kKs16; ++s) {
          nx = mfma32(qf[s], kb[s % kD], nx);
          if (s + kD < kKs16) kb[s % kD] = row_frag(buf, col, g, s + kD);
          if (s >= 2 && s < 34 && (s & 1) == 0) piece((s - 2) >> 1, p_whole, p_t, p_there);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
#pragma unroll
        for (int v = 0; v < 16; ++v) piece(v, p_whole, p_t, p_there);
      }
    }
    if (i > 0) {
      const float w = pair_sum(sum[0] + sum[1]);
      s_w[wave][((i - 1) % kChunk) * kStepTok + col] = w;   // both lanes of a token write the same
    }
    if (i < nsteps) {
      int cnt;
      const int t0 = step_tok(i, &cnt);
      p_t = t0 + col;
      p_there = slot0 >= 0;
      p_whole = even && (uint32_t)__ballot(p_there) == 0xffffffffu && t0 + kStepTok - 1 <= sr.pos0 &&
                (window == 0 || t0 > sr.pos0 + sr.n - 1 - window || t0 + kStepTok <= n_sink);
      st = nx;
      slot0 = slot1;
      slot1 = slot_t;
    }
  }
  __syncthreads();
  __builtin_amdgcn_s_waitcnt(0x70 | 0xF00);
  const int c0 = (nsteps - 1) / kChunk * kChunk;
  write_chunk(c0, nsteps, true);
}

// The decay alone (windowed layers, few queries). grid (ceil(max_len / 1024), B)
__global__ void __launch_bounds__(256)
    paged_weight_decay_kernel(const int32_t* __restrict__ seq_len, Pages pg, int max_len, const float* acc_in, float* acc_out,
                              int64_t acc_ld, float decay) {
  const int b = blockIdx.y;
  const int len = (int)min((int64_t)max(seq_len[b], 0), min((int64_t)max_len, pg.ld * (int64_t)pg.size));
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int t = blockIdx.x * 1024 + u * 256 + threadIdx.x;
    if (t < len) acc_out[(int64_t)b * acc_ld + t] = acc_in ? acc_in[(int64_t)b * acc_ld + t] * decay : 0.f;
  }
}

// ------------------------------------------------------------------ many queries
// Workgroup = 256 tokens of one sequence (wave w: 64 of them, rows in registers)
// and a part of its queries, 32 a step through LDS. Step buffers as above.
constexpr int kTokWg = 256;
constexpr int kQTile = 32;

struct Div {   // m / H = (mulhi(m, mul) + m) >> shift
  uint32_t mul;
  int shift;
};

// grid (ceil(max_len / 256), B, parts)
__global__ void __launch_bounds__(256, 1)
    paged_weight_kernel(const uint16_t* __restrict__ q, int64_t q_rs, int64_t q_hs, const float* __restrict__ lse,
                        const uint4* __restrict__ pool, Pages pg, const int32_t* __restrict__ row0,
                        const int32_t* __restrict__ seq_len, int T, int H, Div by_h, int max_rows, int max_len,
                        int window, int n_sink, float scale2, const float* acc_in, float* acc_out, int64_t acc_ld,
                        float decay, float* __restrict__ part) {
  __shared__ __align__(128) uint8_t tiles[kBufs * kTileB];
  __shared__ __align__(16) float s_lse[4][kBufs][64];   // per wave
  const int b = blockIdx.y, parts = gridDim.z;
  const SeqRows sr = seq_rows(row0, seq_len, pg, b, T, max_rows, max_len);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, col = lane & 31, g = lane >> 5;
  const int tb = blockIdx.x * kTokWg;
  if (tb >= sr.len) return;
  const int te = min(tb + kTokWg, sr.len) - 1;             // last token
  // the rows that see any of the tokens, and this part's steps of their queries
  int r_a = max(0, tb - sr.pos0), r_b = sr.n;
  if (window != 0 && tb >= n_sink) r_b = (int)min((int64_t)r_b, max((int64_t)0, (int64_t)te + window - sr.pos0));
  const int m_a = r_a * H, m_b = max(m_a, r_b * H);
  const int steps = (m_b - m_a + kQTile - 1) / kQTile, per = (steps + parts - 1) / parts;
  const int s0 = min((int)blockIdx.z * per, steps), nsteps = min(s0 + per, steps) - s0;
  const int t_of[2] = {tb + wave * 64 + col, tb + wave * 64 + 32 + col};
  float w[2] = {0.f, 0.f}, lost[2] = {0.f, 0.f};           // sums with what their roundings left out
  bool there[2];

  if (nsteps > 0) {
    const uint32_t lds0 = lds_addr(tiles), lse0 = lds_addr(&s_lse[wave][0][0]);
    const float* lrow = lse + (int64_t)sr.first * H;
    auto issue = [&](int i, int buf) {
      const int m0 = m_a + (s0 + i) * kQTile;
      const uint32_t base = lds0 + static_cast<uint32_t>(buf * kTileB);
      // byte offset of query m0 + col (past the last one: it again)
      const int m = min(m0 + col, m_b - 1), r = (int)((__umulhi((uint32_t)m, by_h.mul) + (uint32_t)m) >> by_h.shift);
      const int64_t off = ((int64_t)(sr.first + r) * q_rs + (int64_t)(m - r * H) * q_hs) * 2;
      const uint8_t* qb = reinterpret_cast<const uint8_t*>(q);
      const int lo = (int)(uint32_t)off, hi = (int)(off >> 32);
      lds_load_dwords(lse0 + buf * 256u, lrow + m);
      {
        const int k = lane >> 3;
        const uint64_t o = (uint64_t)(uint32_t)__shfl(lo, wave * 8 + k, 64) | ((uint64_t)(uint32_t)__shfl(hi, wave * 8 + k, 64) << 32);
        lds_load_lanes(base + kTailAt + wave * 1024, qb + o + kPagedVal * 2 + (((lane & 7) ^ k) * 16));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint64_t o = (uint64_t)(uint32_t)__builtin_amdgcn_readlane(lo, wave * 8 + j) |
                           ((uint64_t)(uint32_t)__builtin_amdgcn_readlane(hi, wave * 8 + j) << 32);
        lds_load_row(base + (wave * 8 + j) * kVPitch, lane * 16, qb + o);
      }
    };
    issue(0, 0);
    bf16x8_t kf[2][kKs16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int slot = t_of[h] <= te ? slot_of(pg, pg.table + (int64_t)b * pg.ld, t_of[h]) : -1;
      there[h] = slot >= 0;
      const uint4* kp = pool + (int64_t)max(slot, 0) * kPagedChunks + g;
#pragma unroll
      for (int s = 0; s < kKs16; ++s) kf[h][s] = __builtin_bit_cast(bf16x8_t, kp[2 * s]);
    }
    // 56 of the 72 fragments live in accumulation registers, which the products
    // read as they are; left to the compiler they would be copied out each time
#pragma unroll
    for (int s = 0; s < kKs16; ++s) {
      asm volatile("" : "+a"(kf[1][s]));
      if (s < 20) asm volatile("" : "+a"(kf[0][s]));
    }
    __builtin_amdgcn_s_waitcnt(0x70 | 0xF00);   // vmcnt(0): step 0, the rows
    issue(min(1, nsteps - 1), 1);
    f32x16_t st[2], nx[2];
#pragma unroll
    for (int v = 0; v < 16; ++v) st[0][v] = st[1][v] = 0.f;
    float ls[16], part4[2][4];
#pragma unroll
    for (int v = 0; v < 16; ++v) ls[v] = 0.f;
    int p_m0 = 0;
    bool p_whole = false;
    const int win = window == 0 ? 0x40000000 : window;   // positions are below 2^30
    auto seen_flat = [&](int p, int t) -> bool { return (t <= p) & ((t > p - win) | (t < n_sink)); };
    // one query (register v) of the scores st of the step before
    auto piece = [&](int v, bool whole) {
      bool in = true;
      int p = 0;
      if (!whole) {
        const int m = p_m0 + 8 * (v >> 2) + 4 * g + (v & 3);
        in = m < m_b;
        p = sr.pos0 + (int)((__umulhi((uint32_t)m, by_h.mul) + (uint32_t)m) >> by_h.shift);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float e = __builtin_amdgcn_exp2f(fmaf(st[h][v], scale2, -ls[v] * kLog2e));
        part4[h][v & 3] += whole | (in & seen_flat(p, t_of[h])) ? e : 0.f;
      }
    };
    auto close = [&]() {   // the step's 16 weights join the running sum
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float y = ((part4[h][0] + part4[h][1]) + (part4[h][2] + part4[h][3])) - lost[h];
        const float t = w[h] + y;
        lost[h] = (t - w[h]) - y;
        w[h] = t;
      }
    };
    for (int i = 0; i < nsteps; ++i) {
      __builtin_amdgcn_s_waitcnt(0x70 | 0xF00 | (kLoads + 1));   // step i has landed, step i + 1 need not have
      __syncthreads();                                           // and step i - 1 is read
      issue(min(i + 2, nsteps - 1), (i + 2) % kBufs);
      const uint8_t* buf = tiles + (i % kBufs) * kTileB;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int u = 0; u < 4; ++u) part4[h][u] = 0.f;
      constexpr int kD = 4;
      bf16x8_t qb[kD];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int v = 0; v < 16; ++v) nx[h][v] = 0.f;
#pragma unroll
      for (int s = 0; s < kD; ++s) qb[s] = row_frag(buf, col, g, s);
      __builtin_amdgcn_sched_barrier(0);
      auto products = [&](bool whole) {
#pragma unroll
        for (int s = 0; s < kKs16; ++s) {
          nx[0] = mfma32(qb[s % kD], kf[0][s], nx[0]);
          nx[1] = mfma32(qb[s % kD], kf[1][s], nx[1]);
          if (s + kD < kKs16) qb[s % kD] = row_frag(buf, col, g, s + kD);
          if (s >= 2 && s < 34 && (s & 1) == 0) piece((s - 2) >> 1, whole);
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      if (i == 0 || p_whole) products(true);
      else products(false);
      if (i > 0) close();
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(&s_lse[wave][i % kBufs][8 * u + 4 * g]);
#pragma unroll
        for (int e = 0; e < 4; ++e) ls[4 * u + e] = x[e];
      }
      st[0] = nx[0];
      st[1] = nx[1];
      p_m0 = m_a + (s0 + i) * kQTile;
      const int r0 = (int)((__umulhi((uint32_t)p_m0, by_h.mul) + (uint32_t)p_m0) >> by_h.shift);
      const int r1 = (int)((__umulhi((uint32_t)(p_m0 + kQTile - 1), by_h.mul) + (uint32_t)(p_m0 + kQTile - 1)) >> by_h.shift);
      p_whole = p_m0 + kQTile <= m_b && te <= sr.pos0 + r0 &&
                (window == 0 || tb > sr.pos0 + r1 - window || te < n_sink);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int u = 0; u < 4; ++u) part4[h][u] = 0.f;
#pragma unroll
    for (int v = 0; v < 16; ++v) piece(v, false);
    close();
    __builtin_amdgcn_s_waitcnt(0x70 | 0xF00);   // no load of a repeat is under way when the workgroup ends
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float x = pair_sum(w[h]);
    const float sum = nsteps > 0 && there[h] ? x : 0.f;   // a token without a page receives nothing
    if (g != 0 || t_of[h] > te) continue;
    if (parts > 1)
      part[((int64_t)blockIdx.z * gridDim.y + b) * max_len + t_of[h]] = sum;
    else
      acc_out[(int64_t)b * acc_ld + t_of[h]] = (acc_in ? acc_in[(int64_t)b * acc_ld + t_of[h]] * decay : 0.f) + sum;
  }
}

// grid (ceil(max_len / 256), B)
__global__ void __launch_bounds__(256)
    paged_weight_join_kernel(const float* __restrict__ part, int parts, Pages pg, const int32_t* __restrict__ row0,
                             const int32_t* __restrict__ seq_len, int T, int max_rows, int max_len,
                             const float* acc_in, float* acc_out, int64_t acc_ld, float decay) {
  const int b = blockIdx.y, t = blockIdx.x * 256 + threadIdx.x;
  const SeqRows sr = seq_rows(row0, seq_len, pg, b, T, max_rows, max_len);
  if (t >= sr.len) return;
  float w = 0.f;
  for (int z = 0; z < parts; ++z) w += part[((int64_t)z * gridDim.y + b) * max_len + t];
  acc_out[(int64_t)b * acc_ld + t] = (acc_in ? acc_in[(int64_t)b * acc_ld + t] * decay : 0.f) + w;
}

bool shape_ok(int B, int T, int H, int max_rows, int max_len) {
  return batch_ok(B, T, max_rows, max_len) && H >= 1 && H <= 128 && (int64_t)T * H < (1ll << 30);
}

bool few(int T, int H, int max_rows) { return (int64_t)std::min(max_rows, T) * H <= kMS; }

// Parts of the queries: as many as fill the CUs evenly with the batch's token
// tiles (a part is at least 16 steps, which its rows' loads are worth). 4 x 40
// token tiles of 128 steps: 3 parts (chosen) 216 us, 4 230 us, 5 249 us, 6 223 us.
int parts_of(int B, int T, int H, int max_rows, int max_len) {
  if (few(T, H, max_rows)) return 1;
  const int64_t wgs = (int64_t)B * ((max_len + kTokWg - 1) / kTokWg);
  const int64_t steps = ((int64_t)std::min(max_rows, T) * H + kQTile - 1) / kQTile;
  if (wgs >= 4 * kCus) return 1;
  int best = 1;
  double cost = 1e30;
  for (int p = 1; p <= 64 && (p == 1 || steps / p >= 16); ++p) {
    const double rounds = (double)((wgs * p + kCus - 1) / kCus);
    const double c = rounds * ((double)steps / p + 10.0);    // 10 steps' time to start
    if (c < cost) cost = c, best = p;
  }
  return best;
}

}  // namespace

extern "C" size_t ech_paged_weight_ws_bytes(int B, int T, int H, int max_rows, int max_len) {
  if (!shape_ok(B, T, H, max_rows, max_len)) return 0;
  const size_t parts = (size_t)parts_of(B, T, H, max_rows, max_len);
  return parts == 1 ? 0 : parts * B * max_len * sizeof(float);
}

extern "C" int ech_paged_weight(const void* q, int64_t q_row_stride, int64_t q_head_stride, const float* lse,
                                const void* pool, int64_t n_slots, int page_size, const int32_t* page_table,
                                int64_t pt_ld, const int32_t* row0, const int32_t* seq_len, int B, int T, int H,
                                int max_rows, int max_len, int window, int n_sink, float sm_scale,
                                const float* acc_in, float* acc_out, int64_t acc_ld, float decay, void* ws,
                                size_t ws_bytes, void* stream) {
  if (!pool || !row0 || !seq_len || !acc_out || (T > 0 && (!q || !lse))) return ECH_EINVAL;
  if (!shape_ok(B, T, H, max_rows, max_len) || window < 0 || n_sink < 0 ||
      !pages_ok(n_slots, page_size, page_table, pt_ld) || acc_ld < max_len)
    return ECH_EINVAL;
  if (!(sm_scale == sm_scale) || !(decay == decay) || !aligned16_(q) || !aligned16_(pool) || q_row_stride < 0 ||
      q_head_stride < 0 || q_row_stride % 8 || q_head_stride % 8)
    return ECH_EINVAL;
  const size_t need = ech_paged_weight_ws_bytes(B, T, H, max_rows, max_len);
  if (ws_bytes < need || (need && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u)))) return ECH_EINVAL;
  if (max_len == 0) return ECH_OK;
  if (window >= max_len) window = 0;                       // no position has more tokens behind it
  n_sink = std::min(n_sink, max_len);
  const Pages pg = make_pages(page_table, pt_ld, n_slots, page_size);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const float scale2 = sm_scale * 1.4426950408889634f;
  if (few(T, H, max_rows)) {
    if (window != 0) {
      hipLaunchKernelGGL(paged_weight_decay_kernel, dim3((max_len + 1023) / 1024, B), dim3(256), 0, s, seq_len, pg, max_len,
                         acc_in, acc_out, acc_ld, decay);
      ECH_LAUNCH_CHECK();
      acc_in = acc_out;
      decay = 1.f;
    }
    const bool planned = B <= kCus && plan_fits(B, B, max_len);
    hipLaunchKernelGGL(paged_weight_stream_kernel, dim3(planned ? kCus : B), dim3(256), 0, s,
                       static_cast<const uint16_t*>(q), q_row_stride, q_head_stride, lse,
                       static_cast<const uint8_t*>(pool), pg, row0, seq_len, B, T, H, max_rows, max_len, window, n_sink,
                       scale2, (int)planned, acc_in, acc_out, acc_ld, decay);
    ECH_LAUNCH_CHECK();
    return ECH_OK;
  }
  const int parts = parts_of(B, T, H, max_rows, max_len);
  const Pages hd = make_pages(nullptr, 1, 1, H);
  hipLaunchKernelGGL(paged_weight_kernel, dim3((max_len + kTokWg - 1) / kTokWg, B, parts), dim3(256), 0, s,
                     static_cast<const uint16_t*>(q), q_row_stride, q_head_stride, lse, static_cast<const uint4*>(pool),
                     pg, row0, seq_len, T, H, Div{hd.mul, hd.shift}, max_rows, max_len, window, n_sink, scale2, acc_in,
                     acc_out, acc_ld, decay, static_cast<float*>(ws));
  ECH_LAUNCH_CHECK();
  if (parts > 1) {
    hipLaunchKernelGGL(paged_weight_join_kernel, dim3((max_len + 255) / 256, B), dim3(256), 0, s,
                       static_cast<const float*>(ws), parts, pg, row0, seq_len, T, max_rows, max_len, acc_in, acc_out,
                       acc_ld, decay);
    ECH_LAUNCH_CHECK();
  }
  return ECH_OK;
}
