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
// Weights that are left out are never subtracted: a chunk's sum leaves a row's
// child tokens out from the start, and theirs are added one by one, so no W is
// the small difference of large sums.
#include <algorithm>

#include "common.hpp"
#include "paged.hpp"

namespace {

constexpr int kDraftMost = 256;              // rows of a tree
constexpr int kChunk = 2048;                 // tokens of a row that a wave sums: 32 a lane
constexpr int kPerLane = kChunk / 64;

struct Stat {                                // of a chunk: the weight of its tokens that are no child's, relative
  double sum;                                // to its largest logit, and the first token that has it
  float top;
  int32_t best;
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
  Stat* stats;                               // [T][chunks]
};

__device__ __forceinline__ float value_of(float x) { return x; }
__device__ __forceinline__ float value_of(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
// NaN weighs nothing, an infinite logit counts as the largest finite one.
__device__ __forceinline__ float logit_of(float x) { return fminf(fmaxf(x, -__builtin_inff()), 3.402823466e38f); }

// 2^t for t <= 0, 0 below 2^-1022 and for NaN: the nearest whole number by an
// addition that rounds there, 2^f of the rest by its series (|f| <= 1/2: what
// the twelve terms leave out is below 7e-15), the whole number added to the
// exponent.
__device__ __forceinline__ double pow2(double t) {
  constexpr double kRound = 6755399441055744.0;            // 1.5 x 2^52
  const double z = t + kRound, f = t - (z - kRound);
  double p = 4.4455382718708100e-10;                       // ln(2)^k / k!, k = 11 .. 0
  p = p * f + 7.0549116208011210e-09;
  p = p * f + 1.0178086009239699e-07;
  p = p * f + 1.3215486790144309e-06;
  p = p * f + 1.5252733804059841e-05;
  p = p * f + 1.5403530393381608e-04;
  p = p * f + 1.3333558146428443e-03;
  p = p * f + 9.6181291076284772e-03;
  p = p * f + 5.5504108664821580e-02;
  p = p * f + 2.4022650695910071e-01;
  p = p * f + 6.9314718055994531e-01;
  p = p * f + 1.0;
  const long long bits = __double_as_longlong(p) + ((long long)(int)__double_as_longlong(z) << 52);
  return t > -1022.0 ? __longlong_as_double(bits) : 0.0;
}
__device__ __forceinline__ double weight_of(float x, float top, double inv_t) { return pow2(((double)x - (double)top) * inv_t); }

// log2(e) / temperature; not above 0 (or NaN): 0, and the call is greedy there.
__device__ __forceinline__ bool greedy_at(const float* temperature, int b, double* inv_t) {
  const float t = temperature ? temperature[b] : 1.f;
  *inv_t = t > 0.f ? 1.4426950408889634 / (double)t : 0.0;
  return !(t > 0.f);
}
__device__ __forceinline__ double unit_of(float u) {       // into [0, 1)
  return (double)fminf(fmaxf(u, 0.f), 0.99999994f);
}
__device__ __forceinline__ int parent_at(const int32_t* parent, int r0, int i) {   // -1: none, or one not before it
  if (!parent) return i - 1;
  const int p = parent[r0 + i];
  return p < i ? max(p, -1) : -1;
}

// Values before the row's first that its first chunk begins with: chunks begin at
// multiples of 16 bytes.
template <typename E>
__device__ __forceinline__ int lead_of(const E* row) {
  return (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(E));
}

__device__ __forceinline__ float lanes_fmax(float x) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor(x, d, 64));
  return x;
}
__device__ __forceinline__ int lanes_min(int x) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x = min(x, __shfl_xor(x, d, 64));
  return x;
}
__device__ __forceinline__ double lanes_sum(double x) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, 64);
  return x;
}
__device__ __forceinline__ double lanes_scan_f64(double x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_up(x, d, 64);
    if (lane >= d) x += o;
  }
  return x;
}

// One chunk of one row, by one wave: its largest logit, and greedy the first
// token that has it, else the weights' sum without the row's child tokens.
template <typename E>
__device__ __forceinline__ void sum_chunk(const Verify<E>& a, int b, int r0, int n, int i, int chunk, int lane) {
  constexpr int kPiece = 16 / sizeof(E);                   // values of a 16-byte load
  const E* row = a.logits + (int64_t)(r0 + i) * a.ld;
  const int e0 = chunk * kChunk - lead_of(row);            // the chunk's first value (may lie before the row)
  if (e0 >= a.V) return;                                   // a row that begins early needs one chunk less
  double inv_t;
  const bool greedy = greedy_at(a.temperature, b, &inv_t);
  float x[kPerLane];
  if (e0 >= 0 && e0 + kChunk <= a.V) {
#pragma unroll
    for (int k = 0; k < kPerLane / kPiece; ++k) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + e0 + (k * 64 + lane) * kPiece);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        if constexpr (sizeof(E) == 2) x[k * kPiece + j] = __uint_as_float(j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
        else x[k * kPiece + j] = __uint_as_float(w[j]);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPerLane / kPiece; ++k)
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        const int e = e0 + (k * 64 + lane) * kPiece + j;
        x[k * kPiece + j] = e >= 0 && e < a.V ? value_of(row[e]) : -__builtin_inff();
      }
  }
  float top = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    x[j] = logit_of(x[j]);
    top = fmaxf(top, x[j]);
  }
  top = lanes_fmax(top);
  int best = -1;
  double sum = 0.0;
  if (greedy) {
    int at = INT32_MAX;
#pragma unroll
    for (int j = kPerLane - 1; j >= 0; --j)
      if (x[j] == top) at = e0 + (j / kPiece * 64 + lane) * kPiece + j % kPiece;
    best = top == -__builtin_inff() ? -1 : lanes_min(at);
  } else {
    for (int j0 = a.parent ? 0 : i + 1; j0 < (a.parent ? n : min(i + 2, n)); j0 += 64) {
      const int j = j0 + lane;
      const int tok = j < n && parent_at(a.parent, r0, j) == i ? a.tokens[r0 + j] : -1;
      unsigned long long hit = __ballot(tok >= max(e0, 0) && tok < min(e0 + kChunk, a.V));
      while (hit != 0ull) {
        const int rel = __builtin_amdgcn_readlane(tok, __builtin_ctzll(hit)) - e0;
        hit &= hit - 1;
        const int at = rel / (64 * kPiece) * kPiece + rel % kPiece;
        const bool mine = rel / kPiece % 64 == lane;
#pragma unroll
        for (int z = 0; z < kPerLane; ++z) x[z] = mine && z == at ? -__builtin_inff() : x[z];
      }
    }
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) sum += weight_of(x[j], top, inv_t);
    sum = lanes_sum(sum);
  }
  if (lane == 0) a.stats[(int64_t)(r0 + i) * a.chunks + chunk] = Stat{sum, top, best};
}

// Every chunk of every row, a wave each: grid (x, y) of ceil(T chunks / 4)
// workgroups or a few more.
constexpr int kStatsX = 1 << 22;
template <typename E>
__global__ void __launch_bounds__(256) draft_stats_kernel(Verify<E> a) {
  const int64_t id = ((int64_t)blockIdx.y * kStatsX + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = threadIdx.x & 63;
  const int t = (int)((uint32_t)id / (uint32_t)a.chunks);  // T chunks < 2^31
  if (t >= a.T || t < a.row0[0]) return;
  int b = 0;                                               // as many sequences as end at or before t precede it
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int c = (int)__popcll(__ballot(b0 + lane < a.B && a.row0[b0 + lane + 1] <= t));
    b += c;
    if (c < 64) break;
  }
  if (b >= a.B) return;
  const int r0 = max(a.row0[b], 0), n = min(min(a.row0[b + 1], a.T) - r0, a.max_rows);
  if (t - r0 >= n || t < r0) return;
  sum_chunk(a, b, r0, n, t - r0, (int)((uint32_t)id - (uint32_t)t * (uint32_t)a.chunks), lane);
}

constexpr int kWalkThreads = 1024, kWalkWaves = kWalkThreads / 64;

// The first thread up to which more than `aim` of the threads' values lies, in
// thread order and behind `before`: found(what lies before its value) is called
// there. Returns before + all values. A thread begins where the one before it
// ends, to the bit, so no aim below the end falls between two. Call from all
// threads.
template <typename F>
__device__ __forceinline__ double find_place(double x, double before, double aim, double* scratch, int* s_win, const F& found) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const double incl = lanes_scan_f64(x, lane);
  const double up = __shfl_up(incl, 1, 64);
  if (lane == 63) scratch[wave] = incl;
  if (tid == 0) *s_win = INT32_MAX;
  __syncthreads();
  double base = before, all = before;
#pragma unroll
  for (int w = 0; w < kWalkWaves; ++w) {
    const double s = scratch[w];
    if (w < wave) base += s;
    all += s;
  }
  const double from = lane == 0 ? base : base + up;
  const bool here = from <= aim && aim < base + incl;      // rounding may make it several
  if (here) atomicMin(s_win, tid);
  __syncthreads();
  if (here && *s_win == tid) found(from);
  __syncthreads();
  return all;
}

struct End {                                 // where a sequence's branch ends
  int32_t row, tried;                        // its row among the batch's (-1: nothing to draw); a chain's draft was tried
  float top;
  int32_t spare;
  double total;                              // the row's weight
};

// The token drawn from a row's weights: chunk_sum(c) and weight(token) say them.
// -1 where nothing weighs. s_int: two words of LDS. Call from all threads.
template <typename C, typename W>
__device__ __forceinline__ int pick(int chunks, int lead, int V, double u, const C& chunk_sum, const W& weight, double* scratch,
                                    int* s_int, double* s_before) {
  const int tid = threadIdx.x;
  int *const s_at = s_int, *const s_win = s_int + 1;
  if (tid == 0) *s_at = -1;
  double total = 0.0;                                      // the chunks' sum first: the aim needs it
  for (int c0 = 0; c0 < chunks; c0 += kWalkThreads)
    total = find_place(c0 + tid < chunks ? chunk_sum(c0 + tid) : 0.0, total, -1.0, scratch, s_win, [](double) {});
  if (!(total > 0.0)) return -1;
  const double aim = u * total;                            // < total, since u < 1
  double before = 0.0;
  for (int c0 = 0; c0 < chunks; c0 += kWalkThreads)
    before = find_place(c0 + tid < chunks ? chunk_sum(c0 + tid) : 0.0, before, aim, scratch, s_win, [&](double at) {
      *s_at = c0 + tid;
      *s_before = at;
    });
  const int chunk = *s_at;
  const double aim_in = aim - *s_before;
  __syncthreads();
  if (tid == 0) *s_at = -1;
  __syncthreads();
  constexpr int kEach = kChunk / kWalkThreads;             // consecutive tokens of a thread
  const int e0 = chunk * kChunk - lead + tid * kEach;
  double w[kEach], mine = 0.0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    w[j] = e0 + j >= 0 && e0 + j < V ? weight(e0 + j) : 0.0;
    mine += w[j];
  }
  int last = -1;                                           // where rounding leaves none: the last that weighs
#pragma unroll
  for (int j = 0; j < kEach; ++j)
    if (w[j] > 0.0) last = e0 + j;
  (void)find_place(mine, 0.0, aim_in, scratch, s_win, [&](double at) {
    int here = last;
    for (int j = kEach - 1; j >= 0; --j) {
      double upto = at;
      for (int k = 0; k <= j; ++k) upto += w[k];
      if (upto > aim_in) here = e0 + j;
    }
    *s_at = here;
  });
  if (*s_at < 0) {
    __syncthreads();
    atomicMax(s_at, last);
    __syncthreads();
  }
  return *s_at;
}

// A sequence's branch and (without a draft) its next token: a workgroup each.
// Its rows' sums are joined, a wave a row; whether a row's token passes depends on
// its siblings before it alone, so all are decided at once, and the branch follows
// each node's first child that passed.
template <typename E>
__global__ void __launch_bounds__(kWalkThreads)
    draft_walk_kernel(Verify<E> a, int32_t* __restrict__ kept, int32_t* __restrict__ n_kept, int32_t* __restrict__ next,
                      End* __restrict__ ends) {
  __shared__ double s_base[kDraftMost], s_w[kDraftMost], scratch[kWalkWaves], s_before;
  __shared__ float s_top[kDraftMost];
  __shared__ int s_best[kDraftMost], s_par[kDraftMost], s_tok[kDraftMost], s_next[kDraftMost];
  __shared__ int s_end[2], s_int[2];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r0 = min(max(a.row0[b], 0), a.T), n = min(min(max(a.row0[b + 1], r0), a.T) - r0, a.max_rows);
  int32_t* const kb = kept + (int64_t)b * a.most;
  if (n <= 0) {
    for (int j = tid; j < a.most; j += kWalkThreads) kb[j] = -1;
    if (tid == 0) {
      n_kept[b] = 0;
      next[b] = -1;
      if (ends) ends[b].row = -1;
    }
    return;
  }
  double inv_t;
  const bool greedy = greedy_at(a.temperature, b, &inv_t);
  float mine = -__builtin_inff();            // the logit of row tid's token, where its parent stands
  if (tid < kDraftMost) {
    const int p = tid < n ? parent_at(a.parent, r0, tid) : -1, tok = tid < n ? a.tokens[r0 + tid] : -1;
    s_par[tid] = p;
    s_tok[tid] = tok;
    s_next[tid] = INT32_MAX;
    if (p >= 0 && tok >= 0 && tok < a.V) mine = logit_of(value_of(a.logits[(int64_t)(r0 + p) * a.ld + tok]));
  }
  for (int i = wave; i < n; i += kWalkWaves) {
    const Stat* st = a.stats + (int64_t)(r0 + i) * a.chunks;
    const int chunks = (a.V + lead_of(a.logits + (int64_t)(r0 + i) * a.ld) + kChunk - 1) / kChunk;
    float top = -__builtin_inff();
    int best = INT32_MAX;
    for (int c = lane; c < chunks; c += 64) {
      const Stat s = st[c];
      if (s.top > top) {
        top = s.top;
        best = s.best;
      }
    }
    const float row_top = lanes_fmax(top);
    double sum = 0.0;
    if (greedy) {
      best = lanes_min(top == row_top && top > -__builtin_inff() ? best : INT32_MAX);
    } else {
      for (int c = lane; c < chunks; c += 64) {
        const Stat s = st[c];
        sum += s.sum * weight_of(s.top, row_top, inv_t);
      }
      sum = lanes_sum(sum);
    }
    if (lane == 0) {
      s_top[i] = row_top;
      s_best[i] = best == INT32_MAX ? -1 : best;
      s_base[i] = sum;
    }
  }
  __syncthreads();
  const int par = tid < n ? s_par[tid] : -1, tok = tid < n ? s_tok[tid] : -1;
  double w = 0.0;
  if (par >= 0) {
    w = weight_of(mine, s_top[par], inv_t);
    if (a.parent)
      for (int j = 0; j < tid; ++j)                        // a sibling's token again
        if (s_par[j] == par && s_tok[j] == tok) w = 0.0;
    s_w[tid] = w;
  }
  __syncthreads();
  if (par >= 0) {
    bool ok;
    if (greedy) {
      ok = tok >= 0 && tok == s_best[par];
    } else {
      double left = s_base[par] + w;
      if (a.parent)
        for (int j = tid + 1; j < n; ++j) left += s_par[j] == par ? s_w[j] : 0.0;
      double bar = unit_of(a.u[r0 + tid]) * left;
      if (a.draft && tok >= 0 && tok < a.V) bar *= (double)fmaxf(a.draft[(int64_t)(r0 + par) * a.draft_ld + tok], 0.f);
      ok = w > 0.0 && bar < w;
    }
    if (ok) atomicMin(&s_next[par], tid);
  }
  __syncthreads();
  if (tid == 0) {
    int at = 0, count = 1;
    kb[0] = 0;
    while (count < a.most && s_next[at] < n) {             // ascends
      at = s_next[at];
      kb[count++] = at;
    }
    n_kept[b] = count;
    s_end[0] = at;
    s_end[1] = count;
  }
  __syncthreads();
  const int at = s_end[0], count = s_end[1];
  for (int j = count + tid; j < a.most; j += kWalkThreads) kb[j] = -1;
  const bool tried = count < a.most;                       // its children, all of them
  const float top = s_top[at];
  if (a.draft) {
    if (tid == 0) {
      const bool child = at + 1 < n;
      ends[b] = End{greedy ? -1 : r0 + at, tried && child, top, 0, s_base[at] + (child ? s_w[at + 1] : 0.0)};
      if (greedy) next[b] = s_best[at];
    }
    return;
  }
  if (greedy) {
    if (tid == 0) next[b] = s_best[at];
    return;
  }
  const E* row = a.logits + (int64_t)(r0 + at) * a.ld;
  const Stat* st = a.stats + (int64_t)(r0 + at) * a.chunks;
  const int lead = lead_of(row), chunks = (a.V + lead + kChunk - 1) / kChunk;
  const int got = pick(
      chunks, lead, a.V, unit_of(a.u[r0]),
      [&](int c) {
        const Stat s = st[c];
        double x = s.sum * weight_of(s.top, top, inv_t);
        if (!tried)
          for (int j = at + 1; j < n; ++j)
            if (s_par[j] == at && s_tok[j] >= 0 && s_tok[j] < a.V && (s_tok[j] + lead) / kChunk == c) x += s_w[j];
        return x;
      },
      [&](int v) {
        bool out = false;
        if (tried)
          for (int j = at + 1; j < n; ++j) out |= s_par[j] == at && s_tok[j] == v;
        return out ? 0.0 : weight_of(logit_of(value_of(row[v])), top, inv_t);
      },
      scratch, s_int, &s_before);
  if (tid == 0) next[b] = got;
}

// What is left of a row behind a draft that did not pass: max(p - q, 0).
template <typename E>
__device__ __forceinline__ double rest_of(const Verify<E>& a, const End& e, double inv_t, int v) {
  const float q = fmaxf(a.draft[(int64_t)e.row * a.draft_ld + v], 0.f);
  const double p = weight_of(logit_of(value_of(a.logits[(int64_t)e.row * a.ld + v])), e.top, inv_t) / e.total;
  return fmax(p - (double)q, 0.0);
}

// Its sums by chunks, a wave each: grid (ceil(chunks / 4), B).
template <typename E>
__global__ void __launch_bounds__(256) draft_rest_kernel(Verify<E> a, const End* __restrict__ ends, double* __restrict__ rest) {
  const int b = blockIdx.y, c = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  const End e = ends[b];
  if (c >= a.chunks || e.row < 0 || !e.tried) return;
  double inv_t;
  (void)greedy_at(a.temperature, b, &inv_t);
  const int e0 = c * kChunk - lead_of(a.logits + (int64_t)e.row * a.ld);
  double sum = 0.0;
  for (int j = lane; j < kChunk; j += 64) {
    const int v = e0 + j;
    if (v >= 0 && v < a.V) sum += rest_of(a, e, inv_t, v);
  }
  sum = lanes_sum(sum);
  if (lane == 0) rest[(int64_t)b * a.chunks + c] = sum;
}

// The next token of chains that were drawn from a draft: a workgroup each.
template <typename E>
__global__ void __launch_bounds__(kWalkThreads)
    draft_pick_kernel(Verify<E> a, const End* __restrict__ ends, const double* __restrict__ rest, int32_t* __restrict__ next) {
  __shared__ double scratch[kWalkWaves], s_before;
  __shared__ int s_int[2];
  const int b = blockIdx.x, tid = threadIdx.x;
  const End e = ends[b];
  if (e.row < 0) return;                                   // no rows, or greedy: written
  double inv_t;
  (void)greedy_at(a.temperature, b, &inv_t);
  const int r0 = min(max(a.row0[b], 0), a.T), n = min(min(max(a.row0[b + 1], r0), a.T) - r0, a.max_rows);
  const E* row = a.logits + (int64_t)e.row * a.ld;
  const Stat* st = a.stats + (int64_t)e.row * a.chunks;
  const int lead = lead_of(row), chunks = (a.V + lead + kChunk - 1) / kChunk;
  const double u = unit_of(a.u[r0]);
  int got = -1;
  if (e.tried)
    got = pick(
        chunks, lead, a.V, u, [&](int c) { return rest[(int64_t)b * a.chunks + c]; },
        [&](int v) { return rest_of(a, e, inv_t, v); }, scratch, s_int, &s_before);
  if (got < 0) {                                           // nothing was tried, or q is nowhere below p
    const int child = e.row + 1 < r0 + n ? a.tokens[e.row + 1] : -1;
    __syncthreads();
    got = pick(
        chunks, lead, a.V, u,
        [&](int c) {
          const Stat s = st[c];
          double x = s.sum * weight_of(s.top, e.top, inv_t);
          if (child >= 0 && child < a.V && (child + lead) / kChunk == c)
            x += weight_of(logit_of(value_of(row[child])), e.top, inv_t);
          return x;
        },
        [&](int v) { return weight_of(logit_of(value_of(row[v])), e.top, inv_t); }, scratch, s_int, &s_before);
  }
  if (tid == 0) next[b] = got;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
int chunks_of(int V) { return (V + 7 + kChunk - 1) / kChunk; }

struct VerifyWs {
  size_t ends, rest, bytes;                  // offsets behind the rows' sums
};
VerifyWs ws_of(int B, int T, int V) {
  VerifyWs w;
  w.ends = up256((size_t)T * chunks_of(V) * sizeof(Stat));
  w.rest = w.ends + up256((size_t)B * sizeof(End));
  w.bytes = w.rest + up256((size_t)B * chunks_of(V) * sizeof(double));
  return w;
}

bool verify_shape_ok(int B, int T, int V, int max_rows, int most) {
  return B >= 1 && B <= 65535 && T >= 0 && V >= 1 && V <= (1 << 24) && max_rows >= 0 && max_rows <= kDraftMost && most >= 1 &&
         (int64_t)T * chunks_of(V) < (1ll << 31) - 4;
}

template <typename E>
int verify_call(const Verify<E>& a, int32_t* kept, int32_t* n_kept, int32_t* next, char* ws, const VerifyWs& w, hipStream_t s) {
  End* ends = a.draft ? reinterpret_cast<End*>(ws + w.ends) : nullptr;
  double* rest = reinterpret_cast<double*>(ws + w.rest);
  const int64_t wgs = ((int64_t)a.T * a.chunks + 3) / 4;
  if (wgs > 0 && a.max_rows > 0) {
    hipLaunchKernelGGL(draft_stats_kernel<E>, dim3((unsigned)std::min<int64_t>(wgs, kStatsX), (unsigned)((wgs + kStatsX - 1) / kStatsX)),
                       dim3(256), 0, s, a);
    ECH_LAUNCH_CHECK();
  }
  hipLaunchKernelGGL(draft_walk_kernel<E>, dim3(a.B), dim3(kWalkThreads), 0, s, a, kept, n_kept, next, ends);
  ECH_LAUNCH_CHECK();
  if (a.draft) {
    hipLaunchKernelGGL(draft_rest_kernel<E>, dim3((a.chunks + 3) / 4, a.B), dim3(256), 0, s, a, ends, rest);
    ECH_LAUNCH_CHECK();
    hipLaunchKernelGGL(draft_pick_kernel<E>, dim3(a.B), dim3(kWalkThreads), 0, s, a, ends, rest, next);
    ECH_LAUNCH_CHECK();
  }
  return ECH_OK;
}

}  // namespace

extern "C" size_t ech_draft_verify_ws_bytes(int B, int T, int V, int max_rows, int most) {
  if (!verify_shape_ok(B, T, V, max_rows, most)) return 0;
  return ws_of(B, T, V).bytes;
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
  const VerifyWs w = ws_of(B, T, V);
  if (ws_bytes < w.bytes || !ws || (reinterpret_cast<uintptr_t>(ws) & 255u)) return ECH_EINVAL;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  char* wp = static_cast<char*>(ws);
  Stat* stats = reinterpret_cast<Stat*>(wp);
  const int chunks = chunks_of(V);
  if (ltype == ECH_LOGIT_BF16)
    return verify_call(Verify<uint16_t>{static_cast<const uint16_t*>(logits), ld, V, chunks, tokens, parent, draft, draft_ld, u,
                                        temperature, row0, B, T, max_rows, most, stats},
                       kept, n_kept, next_token, wp, w, s);
  return verify_call(Verify<float>{static_cast<const float*>(logits), ld, V, chunks, tokens, parent, draft, draft_ld, u,
                                   temperature, row0, B, T, max_rows, most, stats},
                     kept, n_kept, next_token, wp, w, s);
}
