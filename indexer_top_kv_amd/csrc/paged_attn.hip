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

#include "common.hpp"
#include "paged.hpp"

namespace {

typedef __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16 bf16x8_t;
typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16_t;
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef short v4s_t __attribute__((ext_vector_type(4)));
typedef short v8s_t __attribute__((ext_vector_type(8)));

constexpr int kMT = 128;                     // queries per workgroup
constexpr int kStepTok = 32;                 // tokens per step
constexpr int kKs16 = kPagedRow / 16;        // contraction steps of the scores (36)
constexpr int kPitchC = 73;                  // 16-byte pieces per token row in LDS (one spare: bank spread)
constexpr int kPitch = kPitchC * 16;
constexpr int kPos = kStepTok * kPitchC;     // piece positions of a step
constexpr int kTileB = ((kPos + 63) / 64) * 1024;   // bytes of a step's buffer (whole load instructions)
constexpr int kInstr = (kPos + 63) / 64;
constexpr int kPPitch = 80;                  // bytes per query of P in LDS (64 + 16: bank spread)

#define ECH_LDS_PTR(p) ((__attribute__((address_space(3))) void*)(p))

__device__ __forceinline__ bf16x8_t ld_bf16x8(const uint8_t* p) {
  return __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t*>(p));
}

__device__ __forceinline__ f32x16_t mfma32(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// 8 tokens x this lane's column, from two transposed reads of 4 tokens.
__device__ __forceinline__ bf16x8_t ld_tr8(const uint8_t* p0, const uint8_t* p1) {
  const v4s_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s_t*)(p0));
  const v4s_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s_t*)(p1));
  const v8s_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8_t, v);
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

// The tokens a tile of queries at positions [p_lo, p_hi] reads, as up to two
// ranges: [0, n0) and [w0, w1). Steps of 32 tokens run through the first, then
// the second.
struct Ranges {
  int n0, w0, w1, s0, steps;
};
__device__ __forceinline__ Ranges ranges_of(int p_lo, int p_hi, int window, int n_sink) {
  const int end = p_hi + 1;                               // <= len
  const int w0 = window == 0 ? 0 : max(0, p_lo - window + 1);
  Ranges r;
  if (window == 0 || w0 <= n_sink) {                      // one range
    r = Ranges{0, 0, max(end, 0), 0, 0};
  } else {
    r = Ranges{min(n_sink, end), w0, end, 0, 0};
  }
  r.s0 = (r.n0 + kStepTok - 1) / kStepTok;
  r.steps = r.s0 + (r.w1 - r.w0 + kStepTok - 1) / kStepTok;
  return r;
}

// grid (tiles x spans): workgroup = (tile of 128 queries of one sequence, span
// of its steps). With one span it writes out and lse; with several the span's
// maximum, sum and unnormalised output go to the workspace.
__global__ void __launch_bounds__(256, 1)
    paged_attn_kernel(const uint16_t* __restrict__ q, int64_t q_rs, int64_t q_hs, const uint4* __restrict__ pool, Pages pg,
                      const int32_t* __restrict__ row0, const int32_t* __restrict__ seq_len, int B, int T, int H,
                      int max_rows, int max_len, int window, int n_sink, float scale2, int nsp,
                      uint16_t* __restrict__ out, float* __restrict__ lse, float* __restrict__ part_o,
                      float2* __restrict__ part_ml) {
  __shared__ __align__(16) uint8_t tiles[2][kTileB];
  __shared__ __align__(16) uint8_t ps[kMT * kPPitch];
  __shared__ float s_alpha[kMT], s_m[kMT], s_l[kMT];
  __shared__ int s_grow[4], s_poison[4];
  __shared__ int slots[3][kStepTok];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, col = lane & 31, g = lane >> 5;
  int b, mt;
  find_tile(row0, B, T, max_rows, H, kMT, blockIdx.x / nsp, &b, &mt);
  b = __builtin_amdgcn_readfirstlane(b);
  if (b < 0) return;
  mt = __builtin_amdgcn_readfirstlane(mt);
  const int sp = blockIdx.x % nsp;
  const SeqRows sr = seq_rows(row0, seq_len, pg, b, T, max_rows, max_len);
  const int M = sr.n * H;                                  // fits: T H < 2^31 (checked on the host)
  const int m0 = mt * kMT;
  const int r_lo = m0 / H, r_hi = (min(m0 + kMT, M) - 1) / H;
  const Ranges rg = ranges_of(sr.pos0 + r_lo, sr.pos0 + r_hi, window, n_sink);
  const int per = (rg.steps + nsp - 1) / nsp;
  const int step0 = min(sp * per, rg.steps), nsteps = min(step0 + per, rg.steps) - step0;

  // this lane's query of row tile `wave`
  const int m = m0 + wave * 32 + col;
  const bool live = m < M;
  const int mr = live ? m / H : 0, mh = live ? m - mr * H : 0;
  const int p_row = live ? sr.pos0 + mr : -1;
  bf16x8_t qf[kKs16];
  {
    const uint8_t* qp = reinterpret_cast<const uint8_t*>(q + (int64_t)(sr.first + mr) * q_rs + (int64_t)mh * q_hs) + g * 16;
#pragma unroll
    for (int s = 0; s < kKs16; ++s) {
      qf[s] = __builtin_bit_cast(bf16x8_t, u32x4_t{0, 0, 0, 0});
      if (live) qf[s] = ld_bf16x8(qp + s * 32);
    }
  }
  const int32_t* trow = pg.table + (int64_t)b * pg.ld;

  // tokens of step i: [t0, t0 + count)
  auto step_tok = [&](int i, int* count) -> int {
    const int st = step0 + i;
    const int t0 = st < rg.s0 ? st * kStepTok : rg.w0 + (st - rg.s0) * kStepTok;
    *count = min(kStepTok, (st < rg.s0 ? rg.n0 : rg.w1) - t0);
    return t0;
  };
  auto fetch_slot = [&](int i) -> int {
    int cnt;
    const int t0 = step_tok(i, &cnt);
    return lane < cnt ? slot_of(pg, trow, t0 + lane) : -1;
  };
  // Rows of a step whose slots are in slots[si]: direct loads into LDS, one
  // 1 KiB instruction per 64 piece positions; a token without a slot brings
  // slot 0's row, which no query weighs.
  auto issue = [&](int si, int buf) {
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(ECH_LDS_PTR(&tiles[0][0]))) +
                          static_cast<uint32_t>(buf * kTileB);
#pragma unroll
    for (int j = 0; j < (kInstr + 3) / 4; ++j) {
      const int ins = j * 4 + wave;
      const int p = ins * 64 + ln;
      const int t = p / kPitchC, c = p - t * kPitchC;
      if (ins < kInstr && p < kPos && c < kPagedChunks) {
        const uint4* src = pool + (int64_t)max(slots[si][t], 0) * kPagedChunks + c;
        const uint32_t lds = lds0 + static_cast<uint32_t>(ins * 1024);
        asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory", "m0");
      }
    }
  };

  f32x16_t acc[4][4];   // [column tile][row tile]
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[c][r][v] = 0.f;
  float mx = -__builtin_inff(), l = 0.f;   // running maximum of the query, this lane's part of its sum

  if (nsteps > 0) {
    if (wave == 0 && lane < kStepTok) slots[0][lane] = fetch_slot(0);
    __syncthreads();
    issue(0, 0);
    int nxt = wave == 0 && nsteps > 1 ? fetch_slot(1) : -1;
    for (int i = 0; i < nsteps; ++i) {
      __builtin_amdgcn_s_waitcnt(0x70 | 0xF00);   // vmcnt(0): this wave's loads of step i have landed
      if (wave == 0 && lane < kStepTok && i + 1 < nsteps) slots[(i + 1) % 3][lane] = nxt;
      __syncthreads();
      if (i + 1 < nsteps) issue((i + 1) % 3, (i + 1) & 1);
      if (wave == 0 && i + 2 < nsteps) nxt = fetch_slot(i + 2);
      const uint8_t* cur = &tiles[i & 1][0];
      int cnt;
      const int t0 = step_tok(i, &cnt);

      // scores of 32 tokens x this wave's 32 queries
      f32x16_t st;
#pragma unroll
      for (int v = 0; v < 16; ++v) st[v] = 0.f;
      const uint8_t* kr = cur + col * kPitch + g * 16;
#pragma unroll
      for (int s = 0; s < kKs16; ++s) st = mfma32(ld_bf16x8(kr + s * 32), qf[s], st);

      // lane: query col, tokens t0 + 8 (v / 4) + 4 g + v % 4
      float sv[16];
      float tmax = -__builtin_inff();
      bool poison = false;   // a score that does not count is not finite: its row holds infinities or NaN
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int tt = 8 * (v >> 2) + 4 * g + (v & 3);
        const bool ok = slots[i % 3][tt] >= 0 && sees(p_row, t0 + tt, window, n_sink);
        const float x = st[v] * scale2;
        poison |= !ok && !(fabsf(x) < __builtin_inff());
        sv[v] = ok ? x : -__builtin_inff();
        tmax = fmaxf(tmax, sv[v]);
      }
      tmax = pair_max(tmax);
      // the maximum moves only when a step's exceeds it by more than 8: a
      // weight may reach 2^8, and bf16 and fp32 keep their relative precision
      const bool grow = __any(tmax > mx + 8.f);
      const float mn = grow ? fmaxf(mx, tmax) : mx;
      const float ref = mn == -__builtin_inff() ? 0.f : mn;
      const float alpha = exp2f(mx - ref);                  // 0 while nothing was seen
      float psum = 0.f;
      bf16x8_t pb[2];
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const float p = exp2f(sv[v] - ref);
        psum += p;
        pb[v >> 3][v & 7] = (__bf16)p;
      }
      l = l * (grow ? alpha : 1.f) + psum;
      mx = mn;
      uint8_t* pw = ps + (wave * 32 + col) * kPPitch + g * 16;
      *reinterpret_cast<u32x4_t*>(pw) = __builtin_bit_cast(u32x4_t, pb[0]);
      *reinterpret_cast<u32x4_t*>(pw + 32) = __builtin_bit_cast(u32x4_t, pb[1]);
      if (g == 0) s_alpha[wave * 32 + col] = alpha;
      const bool any_poison = __any(poison);
      if (lane == 0) {
        s_grow[wave] = grow;
        s_poison[wave] = any_poison;
      }
      __syncthreads();

#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (s_grow[r]) {
          const float a = s_alpha[r * 32 + col];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            asm volatile("" : "+a"(acc[c][r]));
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[c][r][v] *= a;
            asm volatile("" : "+a"(acc[c][r]));
          }
        }
      }
      if (s_poison[0] | s_poison[1] | s_poison[2] | s_poison[3]) {
        // A weight of zero must add nothing, but 0 x inf is NaN: values that
        // are not finite become 0 in this wave's columns of the step. A query
        // that sees such a row has a score, so a weight, that is NaN already.
        for (int x = lane; x < kStepTok * 16; x += 64) {
          uint16_t* e = reinterpret_cast<uint16_t*>(&tiles[i & 1][0] + (x >> 4) * kPitch + wave * 256 + (x & 15) * 16);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if ((e[j] & 0x7f80u) == 0x7f80u) e[j] = 0;
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
      // O^T += V^T P^T, contraction order of a lane's 16 scores: tokens
      // {16 c + 4 g .. +3, 16 c + 8 + 4 g .. +3} for half c
      bf16x8_t pf[2][4];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) pf[c][r] = ld_bf16x8(ps + (r * 32 + col) * kPPitch + c * 32 + g * 16);
      const uint8_t* vb = cur + (4 * g + ((lane & 15) >> 2)) * kPitch + wave * 256 + ((lane >> 4) & 1) * 32 + 8 * (lane & 3);
#pragma unroll
      for (int ct = 0; ct < 4; ++ct)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const bf16x8_t vf = ld_tr8(vb + 16 * c * kPitch + ct * 64, vb + (16 * c + 8) * kPitch + ct * 64);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[ct][r] = mfma32(vf, pf[c][r], acc[ct][r]);
        }
    }
  }

  l = pair_sum(l);
  if (g == 0) {
    s_m[wave * 32 + col] = mx;
    s_l[wave * 32 + col] = l;
  }
  const int64_t mg0 = (int64_t)sr.first * H + m0;          // first query among the batch's (row, head) pairs
  if (nsp == 1) {
    __syncthreads();
    if (lse && live && g == 0)
      lse[mg0 + wave * 32 + col] = l == 0.f ? -__builtin_inff() : (mx + log2f(l)) * 0.69314718055994531f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int mm = r * 32 + col;
      const float sl = s_l[mm];
      const float inv = sl == 0.f ? 0.f : 1.f / sl;
      if (m0 + mm < M) {
        uint16_t* o = out + (mg0 + mm) * kPagedVal + wave * 128 + 4 * g;
#pragma unroll
        for (int ct = 0; ct < 4; ++ct)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 bf16x4_t;
            bf16x4_t x;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = (__bf16)(acc[ct][r][4 * j + e] * inv);
            *reinterpret_cast<uint2*>(o + ct * 32 + 8 * j) = __builtin_bit_cast(uint2, x);
          }
      }
    }
    return;
  }
  const int64_t MT_all = (int64_t)T * H;
  if (live && g == 0) part_ml[sp * MT_all + mg0 + wave * 32 + col] = make_float2(mx, l);
  if (nsteps == 0) return;                                  // its (-inf, 0) says so
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int mm = r * 32 + col;
    if (m0 + mm < M) {
      float* o = part_o + (sp * MT_all + mg0 + mm) * kPagedVal + wave * 128 + 4 * g;
#pragma unroll
      for (int ct = 0; ct < 4; ++ct)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<f32x4_t*>(o + ct * 32 + 8 * j) =
              f32x4_t{acc[ct][r][4 * j], acc[ct][r][4 * j + 1], acc[ct][r][4 * j + 2], acc[ct][r][4 * j + 3]};
    }
  }
}

// out and lse of every query from its spans' partials, in span order.
// grid (T H), 128 threads: four value columns each.
__global__ void __launch_bounds__(128)
    paged_attn_merge_kernel(const float* __restrict__ part_o, const float2* __restrict__ part_ml,
                            const int32_t* __restrict__ row0, int B, int T, int H, int nsp, uint16_t* __restrict__ out,
                            float* __restrict__ lse) {
  const int64_t mg = blockIdx.x;
  const int row = (int)(mg / H);
  if (row < row0[0] || row >= row0[B]) return;              // a row of no sequence stays as it was
  const int64_t MT_all = (int64_t)T * H;
  float mx = -__builtin_inff();
  for (int s = 0; s < nsp; ++s) mx = fmaxf(mx, part_ml[s * MT_all + mg].x);
  const float ref = mx == -__builtin_inff() ? 0.f : mx;
  float den = 0.f;
  f32x4_t o = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < nsp; ++s) {
    const float2 ml = part_ml[s * MT_all + mg];
    if (ml.y == 0.f) continue;                              // saw nothing: no output was written
    const float w = exp2f((ml.x == -__builtin_inff() ? 0.f : ml.x) - ref);
    den += w * ml.y;
    const f32x4_t x = *reinterpret_cast<const f32x4_t*>(part_o + (s * MT_all + mg) * kPagedVal + 4 * threadIdx.x);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += w * x[e];
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 bf16x4_t;
  bf16x4_t y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = (__bf16)(o[e] * inv);
  *reinterpret_cast<uint2*>(out + mg * kPagedVal + 4 * threadIdx.x) = __builtin_bit_cast(uint2, y);
  if (lse && threadIdx.x == 0)
    lse[mg] = den == 0.f ? -__builtin_inff() : (ref + log2f(den)) * 0.69314718055994531f;
}

// Upper bound of the batch's tiles: every sequence rounds up once.
int64_t tiles_of(int B, int T, int H, int max_rows) {
  const int64_t per_seq = ((int64_t)std::min(max_rows, T) * H + kMT - 1) / kMT;
  return std::min<int64_t>(B * per_seq, (int64_t)T * H / kMT + B);
}

// Spans per tile: enough workgroups for the 256 CUs, four steps each at least.
int spans_of(int B, int T, int H, int max_rows, int max_len, int window, int n_sink) {
  const int64_t tiles = tiles_of(B, T, H, max_rows);
  int64_t seen = max_len;
  if (window > 0) seen = std::min<int64_t>(seen, (int64_t)window + n_sink + kMT / H + 1);
  const int64_t steps = (seen + kStepTok - 1) / kStepTok + 1;
  const int64_t want = std::min<int64_t>(256 / std::max<int64_t>(tiles, 1), steps / 4);
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, 64));
}

bool shape_ok(int B, int T, int H, int max_rows, int max_len, int window, int n_sink) {
  return batch_ok(B, T, max_rows, max_len) && H >= 1 && H <= 128 && (int64_t)T * H < (1ll << 30) && window >= 0 &&
         n_sink >= 0;
}

}  // namespace

extern "C" size_t ech_paged_attn_ws_bytes(int B, int T, int H, int max_rows, int max_len, int window, int n_sink) {
  if (!shape_ok(B, T, H, max_rows, max_len, window, n_sink)) return 0;
  const size_t nsp = (size_t)spans_of(B, T, H, max_rows, max_len, window, n_sink);
  if (nsp == 1) return 0;
  return nsp * T * H * (kPagedVal * sizeof(float) + sizeof(float2));
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
  const int nsp = spans_of(B, T, H, max_rows, max_len, window, n_sink);
  const int64_t tiles = tiles_of(B, T, H, max_rows);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  float* part_o = static_cast<float*>(ws);
  float2* part_ml = reinterpret_cast<float2*>(part_o + (size_t)nsp * T * H * kPagedVal);
  const Pages pg{page_table, pt_ld, n_slots, page_size};
  hipLaunchKernelGGL(paged_attn_kernel, dim3((unsigned)(tiles * nsp)), dim3(256), 0, s, static_cast<const uint16_t*>(q),
                     q_row_stride, q_head_stride, static_cast<const uint4*>(pool), pg, row0, seq_len, B, T, H, max_rows,
                     max_len, window, n_sink, sm_scale * 1.4426950408889634f, nsp, static_cast<uint16_t*>(out), lse,
                     part_o, part_ml);
  ECH_LAUNCH_CHECK();
  if (nsp > 1) {
    hipLaunchKernelGGL(paged_attn_merge_kernel, dim3((unsigned)((int64_t)T * H)), dim3(kPagedVal / 4), 0, s, part_o,
                       part_ml, row0, B, T, H, nsp, static_cast<uint16_t*>(out), lse);
    ECH_LAUNCH_CHECK();
  }
  return ECH_OK;
}
