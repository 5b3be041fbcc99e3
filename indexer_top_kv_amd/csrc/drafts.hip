// Which drafted tokens the target's probabilities accept, from given random
// numbers, and the token that follows them (ech_draft_verify).
//
//   w(v) = exp((logit(v) - largest) / temperature), in 64 bits throughout: every
//   decision compares a random number with sums of w over the vocabulary
//
// At node r the children c1 < c2 < .. are tried in order: child c of token x
// passes iff u_c W < w(x), W the weight of all tokens but those tried before it.
// Where none passes, the next token is the first up to which more than u W of
// the weight lies, the tried ones left out. A chain that was drawn from q:
// passes iff u q(x) < w(x) / W, else the next token is drawn from max(w / W - q, 0).
//
// A row is summed by chunks, a wave each, and a decision joins its chunks' sums.
// Weights that are left out are never subtracted: a chunk's sum leaves the row's
// child tokens out from the start, and theirs are added one by one, so no W is
// the small difference of large sums.
#include <algorithm>

#include "common.hpp"
#include "paged.hpp"

namespace {

constexpr int kDraftMost = 256;              // rows of a tree
constexpr int kGroups = kDraftMost / 64;     // of a tree's rows, one a lane
// Tokens that a wave sums, in four loads of 16 bytes a lane: 2048 of bf16, 1024 of
// fp32 (2048 of these take 100 registers and leave four waves for a SIMD: 64 trees of
// 60 rows, 60000 tokens 62 us, with 1024 57; 11 of 34 rows, 67320 tokens 39.4, 38.3).
template <typename E>
constexpr int kChunk = 4 * 64 * 16 / (int)sizeof(E);
constexpr int kLeast = kChunk<float>;
template <typename E>
constexpr int kPerLane = kChunk<E> / 64;
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

struct Stat {                                // of a chunk: the weight of its tokens that are no child's, relative
  double sum;                                // to its largest logit, and (greedy) the first token that has it
  float top;
  int32_t best;
};
struct Place {                               // a branch so far: its last row, how many it has, whether it ends there
  int32_t at, count, ended, spare;
};
struct End {                                 // where a drawn chain's branch ends: its row among the batch's (-1: nothing
  int32_t row, tried;                        // to draw), whether a draft was rejected there, its largest logit and 1 / W
  float top;
  int32_t spare;
  double inv;
};

// What a call works on.
template <typename E>
struct Verify {
  const E* logits;
  int64_t ld;
  int V, chunks;                             // chunks a row takes, wherever it begins
  const int32_t* tokens;
  const int32_t* parent;                     // NULL: a chain
  const float* draft;
  int64_t draft_ld;
  const float* u;
  const float* temperature;
  const int32_t* row0;
  int B, T, max_rows, most;
  int32_t *kept, *n_kept, *next;
  // of the workspace
  Stat* stats;                               // all rows: [T][chunks]; row by row: [2][B][chunks], in turn
  Place* places;                             // row by row: [levels][B]
  End* ends;                                 // drawn: [B], and max(p - q, 0) summed by chunks [B][chunks]
  double* rest;
};

// One sequence: its rows, and how its logits are weighed.
struct Seq {
  int r0, n;
  bool greedy;
  double inv_t, lowest;                      // log2(e) / temperature; a difference of logits whose weight is 0
};
template <typename E>
__device__ __forceinline__ Seq seq_of(const Verify<E>& a, int b) {
  Seq q;
  q.r0 = min(max(a.row0[b], 0), a.T);
  q.n = min(min(max(a.row0[b + 1], q.r0), a.T) - q.r0, a.max_rows);
  const float t = a.temperature ? a.temperature[b] : 1.f;
  q.greedy = !(t > 0.f);
  q.inv_t = fmax(1.4426950408889634 / (double)(q.greedy ? 1.f : t), 1e-290);   // an infinite one: all weigh 1
  q.lowest = -1100.0 / q.inv_t;
  return q;
}

__device__ __forceinline__ float value_of(float x) { return x; }
__device__ __forceinline__ float value_of(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
// NaN weighs nothing, an infinite logit counts as the type's largest finite one.
template <typename E>
constexpr uint32_t kLargest = sizeof(E) == 4 ? 0x7f7fffffu : 0x7f7f0000u;
template <typename E>
__device__ __forceinline__ float logit_at(const E* row, int v) {
  return fminf(fmaxf(value_of(row[v]), -__builtin_inff()), __uint_as_float(kLargest<E>));
}

// 2^((x - top) / temperature in base 2), relative error 4e-11; 0 for -inf and NaN.
// The nearest whole number by an addition that rounds there, 2^f of the rest by a
// minimax polynomial. 64-bit multiply-adds run at the rate of 32-bit ones, and a
// sum of many rows is bound by the instructions, 24 a value, 15 of them here: 3840
// rows of 128000 bf16 logits, every row, take 436 us and 83% of the vector units'
// cycles.
__device__ __forceinline__ double weight_of(double x, double top, const Seq& q) {
  constexpr double kRound = 6755399441055744.0;            // 1.5 x 2^52
  const double d = fmax(x - top, q.lowest), z = fma(d, q.inv_t, kRound), f = fma(d, q.inv_t, kRound - z);
  double p = 1.520193021018367e-05;
  p = fma(p, f, 0.00015469291101901966);
  p = fma(p, f, 0.0013333922529804455);
  p = fma(p, f, 0.0096180272539097);
  p = fma(p, f, 0.055504103534825794);
  p = fma(p, f, 0.2402265119815426);
  p = fma(p, f, 0.6931471807284377);
  p = fma(p, f, 0.9999999999616828);
  return ldexp(p, (int)__double_as_longlong(z));
}
__device__ __forceinline__ double unit_of(float u) {       // into [0, 1)
  return (double)fminf(fmaxf(u, 0.f), 0.99999994f);
}
__device__ __forceinline__ int parent_at(const int32_t* parent, int r0, int i) {   // -1: none, or one not before it
  const int p = parent[r0 + i];
  return p < i ? max(p, -1) : -1;
}
__device__ __forceinline__ float draft_of(float q) { return fmaxf(q, 0.f); }

// Values before the row's first that its first chunk begins with: chunks begin at
// multiples of 16 bytes.
template <typename E>
__device__ __forceinline__ int lead_of(const E* row) {
  return (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(E));
}
template <typename E>
__device__ __forceinline__ int chunks_in(const Verify<E>& a, const E* row) {
  return (a.V + lead_of(row) + kChunk<E> - 1) / kChunk<E>;
}

// Over the wave's lanes in the vector unit: lanes take what is `CTRL` before them,
// and `none` where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t lanes_before(uint32_t x, uint32_t none) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)x, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double lanes_before(double x) {
  return __hiloint2double((int)lanes_before<CTRL, ROWS>((uint32_t)__double2hiint(x), 0u),
                          (int)lanes_before<CTRL, ROWS>((uint32_t)__double2loint(x), 0u));
}
__device__ __forceinline__ double lane_value(double x, int l) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(x), l), __builtin_amdgcn_readlane(__double2loint(x), l));
}
__device__ __forceinline__ double lanes_scan(double x) {   // inclusive
  x += lanes_before<0x111, 0xf>(x);   // row_shr 1, 2, 4, 8
  x += lanes_before<0x112, 0xf>(x);
  x += lanes_before<0x114, 0xf>(x);
  x += lanes_before<0x118, 0xf>(x);
  x += lanes_before<0x142, 0xa>(x);   // row_bcast 15 to rows 1, 3
  x += lanes_before<0x143, 0xc>(x);   // row_bcast 31 to rows 2, 3
  return x;
}
__device__ __forceinline__ double lanes_sum(double x) { return lane_value(lanes_scan(x), 63); }
__device__ __forceinline__ float lanes_top(float x) {
  constexpr uint32_t kNone = 0xff800000u;   // -inf
  auto with = [&](uint32_t o) { x = fmaxf(x, __uint_as_float(o)); };
  with(lanes_before<0x111, 0xf>(__float_as_uint(x), kNone));
  with(lanes_before<0x112, 0xf>(__float_as_uint(x), kNone));
  with(lanes_before<0x114, 0xf>(__float_as_uint(x), kNone));
  with(lanes_before<0x118, 0xf>(__float_as_uint(x), kNone));
  with(lanes_before<0x142, 0xa>(__float_as_uint(x), kNone));
  with(lanes_before<0x143, 0xc>(__float_as_uint(x), kNone));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), 63));
}
__device__ __forceinline__ int lanes_least(int x) {
  auto with = [&](uint32_t o) { x = min(x, (int)o); };
  with(lanes_before<0x111, 0xf>((uint32_t)x, INT32_MAX));
  with(lanes_before<0x112, 0xf>((uint32_t)x, INT32_MAX));
  with(lanes_before<0x114, 0xf>((uint32_t)x, INT32_MAX));
  with(lanes_before<0x118, 0xf>((uint32_t)x, INT32_MAX));
  with(lanes_before<0x142, 0xa>((uint32_t)x, INT32_MAX));
  with(lanes_before<0x143, 0xc>((uint32_t)x, INT32_MAX));
  return __builtin_amdgcn_readlane(x, 63);
}

// A chunk of a row from value e0, a multiple of 16 bytes, on: lane l holds, in
// pieces of 16 bytes, the values e0 + (64 k + l) kPiece .. of piece k. They stay
// as they are in memory (16 registers, which leaves room for more waves); what
// lies outside of the row is -inf.
template <typename E>
struct Chunk {
  static constexpr int kPiece = 16 / sizeof(E), kPieces = kPerLane<E> / kPiece;
  u32x4_t raw[kPieces];
  // the j-th value of this lane, and the token it is of
  __device__ __forceinline__ float value(int j) const {
    const uint32_t w = raw[j / kPiece][j % kPiece * (int)sizeof(E) / 4];
    if constexpr (sizeof(E) == 4) return __uint_as_float(w);
    else return __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
  }
  // those of `out` (a bit a value) -> -inf, infinite ones -> the largest finite
  __device__ __forceinline__ void mend(uint32_t out) {
    constexpr uint32_t kAll = sizeof(E) == 4 ? 0xffffffffu : 0xffffu;
#pragma unroll
    for (int j = 0; j < kPerLane<E>; ++j) {
      const int sh = sizeof(E) == 2 && (j & 1) ? 16 : 0;
      const uint32_t w = raw[j / kPiece][j % kPiece * (int)sizeof(E) / 4], v = w >> sh & kAll;
      const uint32_t inf = sizeof(E) == 4 ? 0x7f800000u : 0x7f80u, low = inf | (kAll ^ kAll >> 1);
      const uint32_t to = (out >> j) & 1u ? low : v == inf ? inf - 1u : v;
      raw[j / kPiece][j % kPiece * (int)sizeof(E) / 4] = (w & ~(kAll << sh)) | to << sh;
    }
  }
  static __device__ __forceinline__ int token(int e0, int j, int lane) { return e0 + (j / kPiece * 64 + lane) * kPiece + j % kPiece; }
  __device__ __forceinline__ void load(const E* row, int V, int e0, int lane) {
    const bool inside = e0 >= 0 && e0 + kChunk<E> <= V;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int e = e0 + (k * 64 + lane) * kPiece;
      if (inside || (e >= 0 && e + kPiece <= V)) {
        raw[k] = *reinterpret_cast<const u32x4_t*>(row + e);
      } else {
        raw[k] = sizeof(E) == 4 ? 0xff800000u : 0xff80ff80u;
        if (e + kPiece > 0 && e < V) {                     // a piece that the row's ends cut
#pragma unroll
          for (int j = 0; j < kPiece; ++j)
            if (e + j >= 0 && e + j < V) {
              if constexpr (sizeof(E) == 4) raw[k][j] = __float_as_uint(row[e + j]);
              else raw[k][j / 2] = j & 1 ? (raw[k][j / 2] & 0xffffu) | (uint32_t)row[e + j] << 16
                                         : (raw[k][j / 2] & 0xffff0000u) | (uint32_t)row[e + j];
            }
        }
      }
    }
  }
};

// The sums of a chunk of row i of a sequence, from its values (the first of them
// e0), by one wave.
template <typename E>
__device__ __forceinline__ void sum_chunk(const Verify<E>& a, const Seq& q, int i, int e0, Chunk<E>& x, Stat* to, int lane) {
  using C = Chunk<E>;
  float top = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < kPerLane<E>; ++j) top = fmaxf(top, x.value(j));   // passes over NaN
  top = lanes_top(top);
  const bool infinite = top == __builtin_inff();
  if (infinite) top = __uint_as_float(kLargest<E>);
  int best = -1;
  double sum = 0.0;
  if (q.greedy) {
    int at = INT32_MAX;
#pragma unroll
    for (int j = kPerLane<E> - 1; j >= 0; --j)
      if (x.value(j) >= top) at = C::token(e0, j, lane);
    best = top == -__builtin_inff() ? -1 : lanes_least(at);
  } else {
    uint32_t out = 0;                                      // child tokens among this lane's values
    const int first = a.parent ? 0 : i + 1, end = a.parent ? q.n : min(i + 2, q.n);
    for (int j0 = first; j0 < end; j0 += 64) {
      const int j = min(j0 + lane, end - 1), t = a.tokens[q.r0 + j];
      const int tok = j0 + lane < end && (!a.parent || parent_at(a.parent, q.r0, j) == i) ? t : -1;
      unsigned long long hit = __ballot(tok >= max(e0, 0) && tok < min(e0 + kChunk<E>, a.V));
      while (hit != 0ull) {
        const int rel = __builtin_amdgcn_readlane(tok, __builtin_ctzll(hit)) - e0;
        hit &= hit - 1;
        const int at = rel / (64 * C::kPiece) * C::kPiece + rel % C::kPiece;
        out |= rel / C::kPiece % 64 == lane ? 1u << at : 0u;
      }
    }
    if (infinite || __any(out != 0u)) x.mend(out);
#pragma unroll
    for (int k = 0; k < C::kPieces; ++k) asm volatile("" : "+v"(x.raw[k]));   // unpacked again, not kept unpacked
    if (top > -__builtin_inff()) {
#pragma unroll
      for (int j = 0; j < kPerLane<E>; ++j) sum += weight_of(x.value(j), top, q);
    }
    sum = lanes_sum(sum);
  }
  if (lane == 0) *to = Stat{sum, top, best};
}

// A row's chunks joined: its largest logit; greedy the first token that has it
// (-1: none), else the weight of its tokens that are no child's. By one wave.
struct Joined {
  float top;
  int best;
  double base;
};
template <typename E>
__device__ __forceinline__ Joined join(const Verify<E>& a, const Seq& q, const E* row, const Stat* st, int lane) {
  const int chunks = chunks_in(a, row);
  const Stat none{0.0, -__builtin_inff(), -1};
  const Stat s0 = lane < chunks ? st[lane] : none;         // the first 64 stay in registers
  float top = s0.top;
  for (int c = 64 + lane; c < chunks; c += 64) top = fmaxf(top, st[c].top);
  Joined r{lanes_top(top), -1, 0.0};
  if (r.top == -__builtin_inff()) return r;
  if (q.greedy) {
    int best = s0.top == r.top ? s0.best : INT32_MAX;
    for (int c = 64 + lane; c < chunks; c += 64)
      if (st[c].top == r.top) best = min(best, st[c].best);
    r.best = lanes_least(best);
  } else {
    double sum = s0.sum * weight_of(s0.top, r.top, q);
    for (int c = 64 + lane; c < chunks; c += 64) sum += st[c].sum * weight_of(st[c].top, r.top, q);
    r.base = lanes_sum(sum);
  }
  return r;
}

// The child that is accepted at row i of a tree or chain, or -1. By one wave. `end`
// (in LDS, or NULL): a chain's largest logit there and its weight with the child's
// too, or greedy its first token.
template <typename E>
__device__ __forceinline__ int decide(const Verify<E>& a, const Seq& q, int i, const Stat* st, int lane, Joined* end = nullptr) {
  const E* row = a.logits + (int64_t)(q.r0 + i) * a.ld;
  if (!a.parent) {
    if (i + 1 >= q.n) {
      if (end) {
        const Joined r = join(a, q, row, st, lane);
        if (lane == 0) *end = r;
      }
      return -1;
    }
    const int tok = a.tokens[q.r0 + i + 1];
    const bool known = tok >= 0 && tok < a.V;
    const float x = known ? logit_at(row, tok) : -__builtin_inff();
    const double u = unit_of(a.u[q.r0 + i + 1]);
    const double drawn = a.draft && known ? (double)draft_of(a.draft[(int64_t)(q.r0 + i) * a.draft_ld + tok]) : 1.0;
    const Joined r = join(a, q, row, st, lane);
    const double w = q.greedy ? 0.0 : weight_of(x, r.top, q);
    if (end && lane == 0) *end = Joined{r.top, r.best, r.base + w};
    if (q.greedy) return known && tok == r.best ? i + 1 : -1;
    return w > 0.0 && u * (r.base + w) * drawn < w ? i + 1 : -1;
  }
  // lane l holds rows l, 64 + l, ..: those that are children of i, their tokens and weights
  unsigned long long kids[kGroups];
  int tok[kGroups];
  float x[kGroups], u[kGroups];
  bool any = false;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    kids[g] = 0ull;
    tok[g] = -1;
    u[g] = 0.f;
    if (g * 64 < q.n) {
      const int j = min(g * 64 + lane, q.n - 1);           // all three asked for at once
      const int up = parent_at(a.parent, q.r0, j), t = a.tokens[q.r0 + j];
      u[g] = a.u[q.r0 + j];
      const bool kid = g * 64 + lane < q.n && up == i;
      kids[g] = __ballot(kid);
      tok[g] = kid ? t : -1;
      any |= kids[g] != 0ull;
    }
  }
  if (!any) return -1;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    x[g] = -__builtin_inff();
    if (g * 64 < q.n && tok[g] >= 0 && tok[g] < a.V) x[g] = logit_at(row, tok[g]);
  }
  const Joined r = join(a, q, row, st, lane);
  if (r.top == -__builtin_inff()) return -1;
  if (q.greedy) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const unsigned long long hit = __ballot(tok[g] == r.best) & kids[g];
      if (hit != 0ull) return g * 64 + __builtin_ctzll(hit);
    }
    return -1;
  }
  double w[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) w[g] = g * 64 < q.n ? weight_of(x[g], r.top, q) : 0.0;
  // a token twice among the children weighs once, at the first
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    for (unsigned long long left = kids[g]; left != 0ull; left &= left - 1) {
      const int l = __builtin_ctzll(left), t = __builtin_amdgcn_readlane(tok[g], l);
#pragma unroll
      for (int h = g; h < kGroups; ++h)
        if (tok[h] == t && (h > g || lane > l)) w[h] = 0.0;
    }
  }
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    for (unsigned long long left = kids[g]; left != 0ull; left &= left - 1) {
      const int l = __builtin_ctzll(left);
      const double mine = lane_value(w[g], l), rest = r.base + lanes_sum((w[0] + w[1]) + (w[2] + w[3]));
      const float here = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(u[g]), l));
      if (mine > 0.0 && unit_of(here) * rest < mine) return g * 64 + l;
      if (lane == l) w[g] = 0.0;
    }
  }
  return -1;
}

// ------------------------------------------------------------------ every row at once
// Every chunk of every row, a wave each: grid (x, y) of ceil(T chunks / 4)
// workgroups or a few more.
constexpr int kStatsX = 1 << 22;
template <typename E>
__global__ void __launch_bounds__(256) draft_stats_kernel(Verify<E> a) {
  const int64_t id = ((int64_t)blockIdx.y * kStatsX + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = threadIdx.x & 63;
  if (id >= (int64_t)a.T * a.chunks) return;               // T chunks < 2^31
  const int t = (int)((uint32_t)id / (uint32_t)a.chunks), chunk = (int)((uint32_t)id - (uint32_t)t * (uint32_t)a.chunks);
  const E* row = a.logits + (int64_t)t * a.ld;
  const int e0 = chunk * kChunk<E> - lead_of(row);            // the chunk's first value (may lie before the row)
  if (e0 >= a.V) return;                                   // a row that begins early needs one chunk less
  Chunk<E> x;
  x.load(row, a.V, e0, lane);                              // on its way while the row's sequence is found
  if (t < a.row0[0]) return;
  int b = 0;                                               // as many sequences as end at or before t precede it
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int c = (int)__popcll(__ballot(b0 + lane < a.B && a.row0[b0 + lane + 1] <= t));
    b += c;
    if (c < 64) break;
  }
  if (b >= a.B) return;
  const Seq q = seq_of(a, b);
  if (t - q.r0 >= q.n || t < q.r0) return;
  sum_chunk(a, q, t - q.r0, e0, x, a.stats + (int64_t)t * a.chunks + chunk, lane);
}

// ------------------------------------------------------------------ row by row
// Level l: what the row of level l - 1 decides, by every wave alike, and the sums
// of the row that follows. grid (ceil(chunks / 4), B).
template <typename E>
__device__ __forceinline__ Place go_on(const Verify<E>& a, const Seq& q, int b, int level, int lane) {
  Place p = a.places[(int64_t)(level - 1) * a.B + b];
  if (p.ended) return p;
  const int next = decide(a, q, p.at, a.stats + ((int64_t)((level - 1) & 1) * a.B + b) * a.chunks, lane);
  return next < 0 ? Place{p.at, p.count, 1, 0} : Place{next, p.count + 1, 0, 0};
}
template <typename E>
__global__ void __launch_bounds__(256) draft_level_kernel(Verify<E> a, int level) {
  const int b = blockIdx.y, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int chunk = blockIdx.x * 4 + wave;
  const Seq q = seq_of(a, b);
  const Place p = level > 0 ? go_on(a, q, b, level, lane) : Place{0, 1, q.n <= 0, 0};
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.places[(int64_t)level * a.B + b] = p;
    if (!p.ended) a.kept[(int64_t)b * a.most + level] = p.at;
  }
  const E* row = a.logits + (int64_t)(q.r0 + p.at) * a.ld;
  const int e0 = chunk * kChunk<E> - lead_of(row);
  if (p.ended || e0 >= a.V) return;
  Chunk<E> x;
  x.load(row, a.V, e0, lane);
  sum_chunk(a, q, p.at, e0, x, a.stats + ((int64_t)(level & 1) * a.B + b) * a.chunks + chunk, lane);
}

// ------------------------------------------------------------------ the branch and its next token
// Where sequence b's branch ends, in every thread: row `at` of it, the `count`-th
// kept. Row by row the levels have found it (levels of them); else WAVES rows are
// decided at a time, a wave each, from the one that the branch has reached on.
// `write`: kept and n_kept leave. `s_end`: of the rows decided last, the first of
// which is `spare`.
template <int WAVES, bool LEVELS, typename E>
__device__ __forceinline__ Place branch(const Verify<E>& a, const Seq& q, int b, int levels, bool write, int* s_next,
                                        Joined* s_end = nullptr) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  int32_t* const kb = a.kept + (int64_t)b * a.most;
  Place p{0, 1, 0, 0};
  if (LEVELS) {
    p = a.places[(int64_t)(levels - 1) * a.B + b];
    if (!p.ended && p.count < a.most) p = go_on(a, q, b, levels, lane);   // levels = max_rows: finds none
  } else {
    if (write && threadIdx.x == 0) kb[0] = 0;
    for (int first = 0;; first = p.at / WAVES * WAVES) {
      if (first + wave < q.n) {
        const int next = decide(a, q, first + wave, a.stats + (int64_t)(q.r0 + first + wave) * a.chunks, lane,
                                s_end ? s_end + wave : nullptr);
        if (lane == 0) s_next[wave] = next;
      }
      __syncthreads();
      p.spare = first;
      while (!p.ended && p.at < first + WAVES) {
        const int next = p.count < a.most ? s_next[p.at - first] : -1;
        if (next < 0) {
          p.ended = 1;
        } else {
          p.at = next;
          if (write && threadIdx.x == 0) kb[p.count] = next;
          ++p.count;
        }
      }
      if (p.ended) break;
      __syncthreads();
    }
  }
  if (write) {
    for (int j = p.count + threadIdx.x; j < a.most; j += WAVES * 64) kb[j] = -1;
    if (threadIdx.x == 0) a.n_kept[b] = p.count;
  }
  return p;
}
template <int WAVES, typename E>
__device__ __forceinline__ void no_rows(const Verify<E>& a, int b) {
  for (int j = threadIdx.x; j < a.most; j += WAVES * 64) a.kept[(int64_t)b * a.most + j] = -1;
  if (threadIdx.x == 0) {
    a.n_kept[b] = 0;
    a.next[b] = -1;
  }
}

constexpr int kPickThreads = 512, kPickWaves = kPickThreads / 64;
struct PickShared {
  double sum[kPickWaves];
  int hit[kPickWaves], last[kPickWaves];
};

// The first token up to which more than u of a row's weight lies (-1: nothing
// weighs). chunk_sum(c) and weight(token) say the weights. Every wave finds the
// chunk alike; its tokens are four a thread. Call from all threads.
template <typename E, typename C, typename W>
__device__ __forceinline__ int pick(int chunks, int lead, int V, double u, const C& chunk_sum, const W& weight, PickShared& sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const double x0 = lane < chunks ? chunk_sum(lane) : 0.0, scan0 = lanes_scan(x0);
  double total = lane_value(scan0, 63);
  for (int c0 = 64; c0 < chunks; c0 += 64) total += lanes_sum(c0 + lane < chunks ? chunk_sum(c0 + lane) : 0.0);
  if (!(total > 0.0)) return -1;
  const double aim = u * total;                            // < total, since u < 1
  double base = 0.0, before = 0.0;
  int chunk = -1;
  for (int c0 = 0; c0 < chunks; c0 += 64) {
    const double x = c0 == 0 ? x0 : c0 + lane < chunks ? chunk_sum(c0 + lane) : 0.0, incl = c0 == 0 ? scan0 : lanes_scan(x);
    const unsigned long long past = __ballot(x > 0.0 && aim < base + incl), some = __ballot(x > 0.0);
    const int l = past != 0ull ? __builtin_ctzll(past) : some != 0ull ? 63 - __builtin_clzll(some) : -1;
    if (l >= 0) {                                          // the last that weighs, should rounding leave none
      chunk = c0 + l;
      before = l == 0 ? base : base + lane_value(incl, l - 1);
    }
    if (past != 0ull) break;
    base += lane_value(incl, 63);
  }
  const double aim_in = aim - before;
  constexpr int kEach = kChunk<E> / kPickThreads;
  const int e0 = chunk * kChunk<E> - lead + tid * kEach;
  double w[kEach], mine = 0.0;
  int last = -1;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    w[j] = e0 + j >= 0 && e0 + j < V ? weight(e0 + j) : 0.0;
    mine += w[j];
    if (w[j] > 0.0) last = e0 + j;
  }
  const double incl = lanes_scan(mine);
  if (lane == 63) sh.sum[wave] = incl;
  __syncthreads();
  double from = 0.0;
#pragma unroll
  for (int z = 0; z < kPickWaves; ++z)
    if (z < wave) from += sh.sum[z];
  const unsigned long long past = __ballot(last >= 0 && aim_in < from + incl), some = __ballot(last >= 0);
  if (lane == 0) {
    sh.hit[wave] = -1;
    sh.last[wave] = -1;
  }
  if (past != 0ull && lane == __builtin_ctzll(past)) {
    double upto = from + (incl - mine);
    int here = last;
#pragma unroll
    for (int j = kEach - 1; j >= 0; --j) {
      double s = upto;
#pragma unroll
      for (int k = 0; k <= j; ++k) s += w[k];
      if (aim_in < s && w[j] > 0.0) here = e0 + j;
    }
    sh.hit[wave] = here;
  }
  if (some != 0ull && lane == 63 - __builtin_clzll(some)) sh.last[wave] = last;
  __syncthreads();
  int got = -1, end = -1;
#pragma unroll
  for (int z = kPickWaves - 1; z >= 0; --z) {
    if (sh.hit[z] >= 0) got = sh.hit[z];
    if (end < 0) end = sh.last[z];
  }
  __syncthreads();                                         // before sh's next use
  return got >= 0 ? got : end;
}

// The next token behind row p.at from its weights, without its children's where
// they were tried.
template <typename E>
__device__ __forceinline__ int pick_row(const Verify<E>& a, const Seq& q, int b, const Place& p, const Stat* st, bool tried, PickShared& sh) {
  const int lane = threadIdx.x & 63, at = p.at;
  const E* row = a.logits + (int64_t)(q.r0 + at) * a.ld;
  const int lead = lead_of(row), chunks = chunks_in(a, row);
  // its children's tokens; those that have one before them among them count once
  unsigned long long kids[kGroups];
  int tok[kGroups];
  double w[kGroups];
  const Joined r = join(a, q, row, st, lane);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    kids[g] = 0ull;
    tok[g] = -1;
    w[g] = 0.0;
    if (g * 64 < q.n) {
      const int j = min(g * 64 + lane, q.n - 1), up = a.parent ? parent_at(a.parent, q.r0, j) : j - 1;
      const int t = a.tokens[q.r0 + j];
      if (g * 64 + lane < q.n && up == at && t >= 0 && t < a.V) {
        tok[g] = t;
        if (!tried) w[g] = weight_of(logit_at(row, t), r.top, q);
      }
      kids[g] = __ballot(tok[g] >= 0);
    }
  }
  if (!tried) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      for (unsigned long long left = kids[g]; left != 0ull; left &= left - 1) {
        const int l = __builtin_ctzll(left), t = __builtin_amdgcn_readlane(tok[g], l);
#pragma unroll
        for (int h = g; h < kGroups; ++h)
          if (tok[h] == t && (h > g || lane > l)) w[h] = 0.0;
      }
    }
  }
  return pick<E>(
      chunks, lead, a.V, unit_of(a.u[q.r0]),
      [&](int c) {
        const Stat s = st[c];
        double x = s.sum * weight_of(s.top, r.top, q);
        if (!tried) {
#pragma unroll
          for (int g = 0; g < kGroups; ++g)
            for (unsigned long long left = kids[g]; left != 0ull; left &= left - 1) {
              const int l = __builtin_ctzll(left);
              if ((__builtin_amdgcn_readlane(tok[g], l) + lead) / kChunk<E> == c) x += lane_value(w[g], l);
            }
        }
        return x;
      },
      [&](int v) {
        bool out = false;
        if (tried) {
#pragma unroll
          for (int g = 0; g < kGroups; ++g)
            for (unsigned long long left = kids[g]; left != 0ull; left &= left - 1)
              out |= __builtin_amdgcn_readlane(tok[g], __builtin_ctzll(left)) == v;
        }
        return out ? 0.0 : weight_of(logit_at(row, v), r.top, q);
      },
      sh);
}

// A workgroup per sequence.
template <typename E, bool LEVELS>
__global__ void __launch_bounds__(kPickThreads) draft_next_kernel(Verify<E> a, int levels) {
  __shared__ int s_next[kPickWaves];
  __shared__ PickShared sh;
  const int b = blockIdx.x, lane = threadIdx.x & 63;
  const Seq q = seq_of(a, b);
  if (q.n <= 0) return no_rows<kPickWaves>(a, b);
  const Place p = branch<kPickWaves, LEVELS>(a, q, b, levels, true, s_next);
  const Stat* st = a.stats + (LEVELS ? (int64_t)((p.count - 1) & 1) * a.B + b : (int64_t)q.r0 + p.at) * a.chunks;
  int got;
  if (q.greedy) got = join(a, q, a.logits + (int64_t)(q.r0 + p.at) * a.ld, st, lane).best;
  else got = pick_row(a, q, b, p, st, p.count < a.most, sh);
  if (threadIdx.x == 0) a.next[b] = got;
}

// ------------------------------------------------------------------ drawn chains
// Behind a draft that did not pass: max(p - q, 0) by chunks, a wave each. Every
// workgroup finds the branch, eight rows at a time; the first of a sequence writes
// it. grid (ceil(chunks / 8), B).
template <typename E>
__device__ __forceinline__ double rest_of(const Seq& q, float x, float draft, float top, double inv) {
  return fmax(fma(weight_of(x, top, q), inv, -(double)draft_of(draft)), 0.0);
}
constexpr int kRestWaves = 8;
template <typename E, bool LEVELS>
__global__ void __launch_bounds__(kRestWaves * 64) draft_rest_kernel(Verify<E> a, int levels) {
  __shared__ int s_next[kRestWaves];
  __shared__ Joined s_end[kRestWaves];
  const int b = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool first = blockIdx.x == 0;
  const Seq q = seq_of(a, b);
  if (q.n <= 0) {
    if (first) {
      no_rows<kRestWaves>(a, b);
      if (threadIdx.x == 0) a.ends[b].row = -1;
    }
    return;
  }
  const Place p = branch<kRestWaves, LEVELS>(a, q, b, levels, first, s_next, s_end);
  const Stat* st = a.stats + (LEVELS ? (int64_t)((p.count - 1) & 1) * a.B + b : (int64_t)q.r0 + p.at) * a.chunks;
  const E* row = a.logits + (int64_t)(q.r0 + p.at) * a.ld;
  Joined r;
  if (LEVELS) {
    r = join(a, q, row, st, lane);
    const int tok = p.at + 1 < q.n ? a.tokens[q.r0 + p.at + 1] : -1;
    if (tok >= 0 && tok < a.V) r.base += weight_of(logit_at(row, tok), r.top, q);
  } else {
    r = s_end[p.at - p.spare];                             // found with the decision
  }
  if (q.greedy) {
    if (first && threadIdx.x == 0) {
      a.next[b] = r.best;
      a.ends[b].row = -1;
    }
    return;
  }
  const bool tried = p.count < a.most && p.at + 1 < q.n;
  const double inv = 1.0 / r.base;
  if (first && threadIdx.x == 0) a.ends[b] = End{q.r0 + p.at, tried, r.top, 0, inv};
  const int chunk = blockIdx.x * kRestWaves + wave, e0 = chunk * kChunk<E> - lead_of(row);
  if (!tried || e0 >= a.V) return;
  constexpr int kPiece = Chunk<E>::kPiece;
  Chunk<E> x;
  x.load(row, a.V, e0, lane);
  if (r.top == __uint_as_float(kLargest<E>)) x.mend(0u);
  const float* draft = a.draft + (int64_t)(q.r0 + p.at) * a.draft_ld;
  double sum = 0.0;
  if (e0 >= 0 && e0 + kChunk<E> <= a.V && (reinterpret_cast<uintptr_t>(draft + e0) & 15u) == 0) {
#pragma unroll
    for (int k = 0; k < kPerLane<E> / 4; ++k) {
      const f32x4_t d = *reinterpret_cast<const f32x4_t*>(draft + e0 + ((k * 4 / kPiece) * 64 + lane) * kPiece + k * 4 % kPiece);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += rest_of<E>(q, x.value(k * 4 + j), d[j], r.top, inv);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPerLane<E>; ++j) {
      const int v = Chunk<E>::token(e0, j, lane);
      if (v >= 0 && v < a.V) sum += rest_of<E>(q, x.value(j), draft[v], r.top, inv);
    }
  }
  sum = lanes_sum(sum);
  if (lane == 0) a.rest[(int64_t)b * a.chunks + chunk] = sum;
}

// The next token of drawn chains: a workgroup each.
template <typename E, bool LEVELS>
__global__ void __launch_bounds__(kPickThreads) draft_pick_kernel(Verify<E> a) {
  __shared__ PickShared sh;
  const int b = blockIdx.x;
  const End e = a.ends[b];
  if (e.row < 0) return;                                   // no rows, or greedy: written
  const Seq q = seq_of(a, b);
  const E* row = a.logits + (int64_t)e.row * a.ld;
  const float* draft = a.draft + (int64_t)e.row * a.draft_ld;
  int got = -1;
  if (e.tried)
    got = pick<E>(
        chunks_in(a, row), lead_of(row), a.V, unit_of(a.u[q.r0]), [&](int c) { return a.rest[(int64_t)b * a.chunks + c]; },
        [&](int v) { return rest_of<E>(q, logit_at(row, v), draft[v], e.top, e.inv); }, sh);
  if (got < 0) {                                           // nothing was tried, or q is nowhere below p
    const int count = a.n_kept[b];
    const Stat* st = a.stats + (LEVELS ? (int64_t)((count - 1) & 1) * a.B + b : (int64_t)e.row) * a.chunks;
    got = pick_row(a, q, b, Place{e.row - q.r0, count, 1, 0}, st, false, sh);
  }
  if (threadIdx.x == 0) a.next[b] = got;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
int chunks_of(int V, int chunk = kLeast) { return (V + 7 + chunk - 1) / chunk; }

// Every row at once reads all of the T rows (1500 values a ns) in two or three
// launches; row by row only the rows of the branches are read, at most about three
// of a sequence's, in a launch (5 us) for each row that a branch may have. Rows of
// 128000 tokens, trees of 60 rows, branches of up to 11: 64 sequences 58 us row by
// row, 337 at once; 8 of them 44 and 59, 4 of them 40 and 36. 64 of 26 rows, 50021
// tokens, branches of up to 10: 56 and 73; 32 of them 49 and 46.
bool row_by_row(int64_t B, int64_t T, int64_t V, int64_t levels) { return (T - 3 * B) * V > levels * 4000000; }
struct Way {
  int levels;                                // 0: at once
  size_t places, ends, rest, bytes;          // offsets behind the sums
};
Way way_of(int B, int T, int V, int max_rows, int most) {
  Way w;
  const int levels = std::max(1, std::min(most, max_rows));
  w.levels = row_by_row(B, T, V, levels) ? levels : 0;
  const size_t rows = w.levels ? (size_t)2 * B : (size_t)T;
  w.places = up256(rows * chunks_of(V) * sizeof(Stat));
  w.ends = w.places + up256((size_t)w.levels * B * sizeof(Place));
  w.rest = w.ends + up256((size_t)B * sizeof(End));
  w.bytes = w.rest + up256((size_t)B * chunks_of(V) * sizeof(double));
  return w;
}

bool verify_shape_ok(int B, int T, int V, int max_rows, int most) {
  return B >= 1 && B <= 65535 && T >= 0 && V >= 1 && V <= (1 << 24) && max_rows >= 0 && max_rows <= kDraftMost && most >= 1 &&
         (int64_t)T * chunks_of(V) < (1ll << 31) - 4;
}

template <typename E, bool LEVELS>
int verify_call(const Verify<E>& a, int levels, hipStream_t s) {
  const dim3 grid((a.chunks + 3) / 4, a.B);
  if (LEVELS) {
    for (int l = 0; l < levels; ++l) {
      hipLaunchKernelGGL(draft_level_kernel<E>, grid, dim3(256), 0, s, a, l);
      ECH_LAUNCH_CHECK();
    }
  } else {
    const int64_t wgs = ((int64_t)a.T * a.chunks + 3) / 4;
    if (wgs > 0 && a.max_rows > 0) {
      hipLaunchKernelGGL(draft_stats_kernel<E>, dim3((unsigned)std::min<int64_t>(wgs, kStatsX), (unsigned)((wgs + kStatsX - 1) / kStatsX)),
                         dim3(256), 0, s, a);
      ECH_LAUNCH_CHECK();
    }
  }
  if (!a.draft) {
    const auto kernel = draft_next_kernel<E, LEVELS>;
    hipLaunchKernelGGL(kernel, dim3(a.B), dim3(kPickThreads), 0, s, a, levels);
    ECH_LAUNCH_CHECK();
    return ECH_OK;
  }
  const auto rest = draft_rest_kernel<E, LEVELS>;
  hipLaunchKernelGGL(rest, dim3((a.chunks + kRestWaves - 1) / kRestWaves, a.B), dim3(kRestWaves * 64), 0, s, a, levels);
  ECH_LAUNCH_CHECK();
  const auto drawn = draft_pick_kernel<E, LEVELS>;
  hipLaunchKernelGGL(drawn, dim3(a.B), dim3(kPickThreads), 0, s, a);
  ECH_LAUNCH_CHECK();
  return ECH_OK;
}

}  // namespace

extern "C" size_t ech_draft_verify_ws_bytes(int B, int T, int V, int max_rows, int most) {
  if (!verify_shape_ok(B, T, V, max_rows, most)) return 0;
  return way_of(B, T, V, max_rows, most).bytes;
}

extern "C" int ech_draft_verify(const void* logits, int ltype, int64_t ld, int V, const int32_t* tokens,
                                const int32_t* row0, const int32_t* parent, const float* draft, int64_t draft_ld,
                                const float* u, const float* temperature, int B, int T, int max_rows, int most,
                                int32_t* kept, int32_t* n_kept, int32_t* next_token, void* ws, size_t ws_bytes,
                                void* stream) {
  if (ltype != ECH_LOGIT_BF16 && ltype != ECH_LOGIT_F32) return ECH_EUNSUPPORTED;
  if (!row0 || !kept || !n_kept || !next_token || (T > 0 && (!logits || !tokens || !u))) return ECH_EINVAL;
  if (!verify_shape_ok(B, T, V, max_rows, most) || ld < V || (draft && (parent || draft_ld < V))) return ECH_EINVAL;
  const size_t size = ltype == ECH_LOGIT_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(logits) % size || reinterpret_cast<uintptr_t>(draft) % 4) return ECH_EINVAL;
  const Way w = way_of(B, T, V, max_rows, most);
  if (ws_bytes < w.bytes || !ws || (reinterpret_cast<uintptr_t>(ws) & 255u)) return ECH_EINVAL;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  char* wp = static_cast<char*>(ws);
  auto call = [&](auto* x) {
    using E = std::remove_const_t<std::remove_pointer_t<decltype(x)>>;
    const Verify<E> a{x, ld, V, chunks_of(V, kChunk<E>), tokens, parent, draft, draft_ld, u, temperature, row0, B, T, max_rows, most, kept,
                      n_kept, next_token, reinterpret_cast<Stat*>(wp), reinterpret_cast<Place*>(wp + w.places),
                      reinterpret_cast<End*>(wp + w.ends), reinterpret_cast<double*>(wp + w.rest)};
    return w.levels ? verify_call<E, true>(a, w.levels, s) : verify_call<E, false>(a, 0, s);
  };
  return ltype == ECH_LOGIT_BF16 ? call(static_cast<const uint16_t*>(logits)) : call(static_cast<const float*>(logits));
}
