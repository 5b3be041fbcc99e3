// Rows that join and leave a resident paged cache: ech_paged_append puts a
// step's new rows into their sequences' pages, ech_paged_evict keeps `keep`
// tokens of each sequence and moves their rows together, ech_paged_accept does
// so with the accepted ones of a step's drafted rows, and ech_paged_copy copies
// pages.
#include <algorithm>

#include "common.hpp"
#include "paged.hpp"

namespace {

// grid (x, y) of ceil(T / 4) workgroups or a few more, 256 threads (x is at most
// kAppendX: a launch has less than 2^32 threads in x). One wave per row, which
// finds its sequence by counting the row ends at or before it, 64 sequences a
// round. Bound by the rows' bytes, or with few rows by the two dependent reads
// (offsets, page) and the launch: 16384 rows of 1152 bytes 5.8 us (6.5 TB/s of reads and writes, a
// part of them from cache), 64 rows 3.1 us.
constexpr int kAppendX = 1 << 22;
__global__ void __launch_bounds__(256)
    paged_append_kernel(uint4* __restrict__ pool, int row16, Pages pg, const int32_t* __restrict__ row0,
                        const int32_t* __restrict__ seq_len, int B, int T, const uint4* __restrict__ rows,
                        int64_t row_stride16, int32_t* __restrict__ status) {
  const int t = (int)(blockIdx.y * kAppendX + blockIdx.x) * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;   // < 2^31
  if (t >= T || t < row0[0]) return;
  // the sequence whose rows end past t: as many as end at or before it precede it
  int b = 0;
  for (int b0 = 0; b0 < B; b0 += 64) {
    const bool before = b0 + lane < B && row0[b0 + lane + 1] <= t;
    const int c = (int)__popcll(__ballot(before));
    b += c;
    if (c < 64) break;
  }
  if (b >= B) return;                                       // behind the last sequence
  const int64_t pos = (int64_t)seq_len[b] - row0[b + 1] + t;   // < seq_len: row0[b + 1] > t
  const int slot = pos >= 0 ? slot_of(pg, pg.table + (int64_t)b * pg.ld, (int)pos) : -1;
  if (slot < 0) {
    if (status && lane == 0) atomicOr(status, ECH_ST_FULL);
    return;
  }
  for (int i = lane; i < row16; i += 64) pool[(int64_t)slot * row16 + i] = rows[(int64_t)t * row_stride16 + i];
}

// ------------------------------------------------------------------ eviction
// A sequence of n > keep tokens keeps its first n_sink, its last n_recent, and
// of the tokens between the `want` = keep - n_sink - n_recent with the largest
// weights, ties to the lower index. The want-th largest key is found digit by
// digit (11, 11 and 10 bits of an order-preserving 32-bit key) from
// histograms; what is above it and the first `ties` of its equals stay. The
// weights are read once (the one-workgroup form) or once per digit from L2
// (the form for long rows); a wave owns consecutive tokens, 64 per register,
// so ranks come from ballots.
constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 2048;
// A bin's count in LDS is kept four times over, lane l adding to the l % 4-th:
// equal keys (zeros, above all) go to one bin, one after the other. 16384 equal
// weights 20 us, with one count 50 us; spread ones 12 us either way.
constexpr int kCopies = 4;
__device__ __forceinline__ void clear_bins(int* hist) {
#pragma unroll
  for (int z = 0; z < kBins * kCopies / kThreads; ++z) hist[z * kThreads + threadIdx.x] = 0;
}
__device__ __forceinline__ void add_to_bin(int* hist, uint32_t bin) {
  atomicAdd(&hist[bin * kCopies + (threadIdx.x & (kCopies - 1))], 1);
}
__device__ __forceinline__ int bin_count(const int* hist, int bin) {
  const int4 v = *reinterpret_cast<const int4*>(hist + bin * kCopies);
  return (v.x + v.y) + (v.z + v.w);
}

// Order of a weight: larger first; NaN above everything, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float x) { return x != x ? 0xffffffffu : ech::ord_key(x); }

__device__ __forceinline__ int digit_shift(int level) { return level == 0 ? 21 : level == 1 ? 10 : 0; }

struct Row {
  int n, lo, hi, want;   // tokens; those between the protected ones are [lo, hi); how many of them stay
};                       // (none are between where n <= keep)
__device__ __forceinline__ Row row_of(const int32_t* seq_len, int b, int max_len, int keep, int n_sink, int n_recent) {
  const int n = min(max(seq_len[b], 0), max_len);
  const bool cut = n > keep;
  return Row{n, cut ? n_sink : 0, cut ? n - n_recent : 0, cut ? keep - n_sink - n_recent : 0};
}

// The sum of one value per wave (the same in all of its lanes), and what the
// waves before this one hold of it. scratch: kWaves; a barrier has to stand
// between two uses. Call from all threads.
__device__ __forceinline__ int waves_sum(int x, int* scratch, int* before) {
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
  if (lane == 0) scratch[wave] = x;
  __syncthreads();
  const int w = lane < kWaves ? scratch[lane] : 0, incl = lanes_scan(w);
  *before = __builtin_amdgcn_readlane(incl, wave) - x;
  return last_lane(incl);
}

// The digit d of descending bins that holds the want-th entry, and how many of
// that bin are wanted. Thread t brings the counts of bins 2047 - 2t and 2046 -
// 2t; out[0] = d, out[1] = rest. Call from all threads.
__device__ __forceinline__ void find_digit(int c0, int c1, int want, int* scratch, int* out) {
  const int incl = lanes_scan(c0 + c1);
  int waves;
  (void)waves_sum(last_lane(incl), scratch, &waves);
  const int before = waves + incl - (c0 + c1);
  const int d0 = kBins - 1 - 2 * (int)threadIdx.x;
  if (before < want && want <= before + c0) {
    out[0] = d0;
    out[1] = want - before;
  } else if (before + c0 < want && want <= before + c0 + c1) {
    out[0] = d0 - 1;
    out[1] = want - before - c0;
  }
  __syncthreads();
}

// A block of KPT * 1024 tokens from t0: wave w owns KPT * 64 consecutive ones,
// register j 64 of them from this token on.
template <int KPT>
__device__ __forceinline__ int base_of(int t0, int j) {
  return t0 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) * (KPT * 64) + j * 64;
}
// This thread's weights of a block (up to max_len, before the length is known),
// and their keys: 0, which no weight has, for a token that is protected or does
// not exist.
template <int KPT>
__device__ __forceinline__ void load_weights(const float* a, int t0, int max_len, float (&x)[KPT]) {
#pragma unroll
  for (int j = 0; j < KPT; ++j) {
    const int t = base_of<KPT>(t0, j) + (int)(threadIdx.x & 63);
    x[j] = t < max_len ? a[t] : 0.f;
  }
}
template <int KPT>
__device__ __forceinline__ void keys_of(const float (&x)[KPT], int t0, const Row& r, uint32_t (&k)[KPT]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int j = 0; j < KPT; ++j) {
    const int t = base_of<KPT>(t0, j) + lane;
    k[j] = (uint32_t)(t - r.lo) < (uint32_t)(r.hi - r.lo) ? weight_key(x[j]) : 0u;
  }
}

// Counts digit `(k >> shift) mod 2^width` of the block's keys whose higher
// digits are `prefix` (first: of all).
template <int KPT>
__device__ __forceinline__ void count_digits(const uint32_t (&k)[KPT], bool first, uint32_t prefix, int shift, int width,
                                             int* hist) {
  const uint32_t mask = (1u << width) - 1u;
  if (first) {
#pragma unroll
    for (int j = 0; j < KPT; ++j)
      if (k[j] != 0) add_to_bin(hist, k[j] >> shift);
  } else {
#pragma unroll
    for (int j = 0; j < KPT; ++j)
      if (k[j] >> (shift + width) == prefix) add_to_bin(hist, (k[j] >> shift) & mask);
  }
}

__device__ __forceinline__ int set_rank(uint64_t set) {   // of this lane: members in lower lanes
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(set >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)set, 0));
}

// The places of one block's kept tokens, put(place, token, weight) each: the
// protected ones' are known; those with keys above thr, and the equals of thr
// while `ties` (less those before the block, ties0) last, go to places at0, at0
// + 1, ... in token order. A workgroup's 16 waves share one CU's issue and its
// instruction cache, and this code runs once: it is kept short (with a branch
// per case 10K cycles at KPT 16).
template <int KPT, class Put>
__device__ __forceinline__ void place_kept(const float* a, const float (&x)[KPT], uint32_t (&k)[KPT], const Row& r,
                                           int t0, uint32_t thr, int ties, int ties0, int at0, int nk, int (*s_cnt)[2],
                                           Put put) {
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
  int gt = 0, eq = 0;
#pragma unroll
  for (int j = 0; j < KPT; ++j) {
    gt += (int)__popcll(__ballot(k[j] > thr));
    eq += (int)__popcll(__ballot(k[j] == thr));
  }
  if (lane == 0) {
    s_cnt[wave][0] = gt;
    s_cnt[wave][1] = eq;
  }
  __syncthreads();
  // the waves before this one, a wave per lane; of equals the first ties - ties0 stay
  const int2 c = lane < wave ? *reinterpret_cast<const int2*>(s_cnt[lane]) : make_int2(0, 0);
  const int gt0 = last_lane(lanes_scan(c.x)), eq0 = last_lane(lanes_scan(c.y));
  int at = at0 + gt0 + min(max(ties - ties0, 0), eq0), left = ties - ties0 - eq0;
#pragma unroll
  for (int j = 0; j < KPT; ++j) {
    asm volatile("" : "+v"(k[j]));   // compared again: the sets, held, would not fit the scalar registers
    const uint64_t tie = __ballot(k[j] == thr), set = __ballot(k[j] > thr) | (tie & __ballot(set_rank(tie) < left));
    const int place = at + set_rank(set);
    if (__builtin_amdgcn_inverse_ballot_w64(set)) put(place, base_of<KPT>(t0, j) + lane, x[j]);
    at += (int)__popcll(set);
    left -= (int)__popcll(tie);
  }
  auto fixed = [&](int from, int to) {
    for (int t = from + (int)threadIdx.x; t < to; t += kThreads) put(t < r.lo ? t : t - r.n + nk, t, a[t]);
  };
  const int end = t0 + KPT * kThreads;
  fixed(t0, min(r.lo, end));
  fixed(max(r.hi, t0), min(r.n, end));
}

// Values from LDS to memory, 16 bytes a thread: src[0 .. n), then `rest` up to
// `all`. src stands as far past a 16-byte boundary as dst: at lead_of(dst).
__device__ __forceinline__ int lead_of(const void* dst) { return (int)((reinterpret_cast<uintptr_t>(dst) >> 2) & 3); }
template <class V>
__device__ __forceinline__ void copy_out(V* dst, const V* src, int n, V rest, int all) {
  typedef V vec_t __attribute__((ext_vector_type(4)));
  const int lead = lead_of(dst);
  for (int i = 4 * (int)threadIdx.x - lead; i < all; i += 4 * kThreads) {
    if (i >= 0 && i + 4 <= n) {
      *reinterpret_cast<vec_t*>(dst + i) = *reinterpret_cast<const vec_t*>(src + i);
    } else if (i >= n && i + 4 <= all) {
      *reinterpret_cast<vec_t*>(dst + i) = vec_t{rest, rest, rest, rest};
    } else {
      for (int e = max(i, 0); e < min(i + 4, all); ++e) dst[e] = e < n ? src[e] : rest;
    }
  }
}

// Rows of at most KPT * 1024 tokens: one workgroup per sequence, its weights in
// registers from the first read on, so acc_out may be acc and len_out seq_len.
// Bound by one CU's issue: of 27K cycles at KPT 16 the weights take 4.7K to
// arrive, each of the three digits 1.4K to 3.5K to count and 1.3K to find, the
// places 6.8K, the writes 2.2K. KPT 4 to 4096 tokens, 16 to 16384, the form
// below for longer rows; 1, 32 and 256 sequences:
//   4096 tokens    KPT 4  6.7, 6.6, 7.2 us      KPT 16     9.3, 9.7, 10.5 us
//   16384 tokens   KPT 16 12.1, 12.7, 16.0 us   long rows  20.8, 22.4, 35.4 us
template <int KPT>
__global__ void __launch_bounds__(kThreads)
    paged_evict_row_kernel(const float* acc, int64_t acc_ld, const int32_t* seq_len, int max_len, int keep, int n_sink,
                           int n_recent, int32_t* __restrict__ kept, float* acc_out, int32_t* len_out) {
  constexpr int kStage = KPT * kThreads + 4, kHist = kBins * kCopies;
  __shared__ __align__(16) int mem[2 * kStage > kHist ? 2 * kStage : kHist];   // the counts, then what is kept
  __shared__ int scratch[kWaves], s_found[2];
  __shared__ __align__(8) int s_cnt[kWaves][2];
  int* const hist = mem;
  const int b = blockIdx.x, tid = threadIdx.x;
  const float* a = acc + (int64_t)b * acc_ld;
  float x[KPT];
  uint32_t k[KPT];
  load_weights<KPT>(a, 0, max_len, x);
  const Row r = row_of(seq_len, b, max_len, keep, n_sink, n_recent);
  keys_of<KPT>(x, 0, r, k);
  uint32_t thr = 0xffffffffu;
  int ties = 0;
  if (r.want > 0) {
    int want = r.want;
    uint32_t prefix = 0;
    for (int level = 0; level < 3; ++level) {
      const int shift = digit_shift(level), width = level == 2 ? 10 : 11;
      clear_bins(hist);
      __syncthreads();
      count_digits<KPT>(k, level == 0, prefix, shift, width, hist);
      __syncthreads();
      find_digit(bin_count(hist, kBins - 1 - 2 * tid), bin_count(hist, kBins - 2 - 2 * tid), want, scratch, s_found);
      prefix = (prefix << width) | (uint32_t)s_found[0];
      want = s_found[1];
      __syncthreads();
    }
    thr = prefix;
    ties = want;
  }
  const int nk = min(r.n, keep);
  int32_t* kb = kept + (int64_t)b * keep;
  float* ao = acc_out ? acc_out + (int64_t)b * acc_ld : nullptr;
  int* const s_kept = mem + lead_of(kb);
  float* const s_out = reinterpret_cast<float*>(mem + kStage) + lead_of(ao);
  place_kept<KPT>(a, x, k, r, 0, thr, ties, 0, r.lo, nk, s_cnt, [&](int place, int t, float v) {
    s_kept[place] = t;
    s_out[place] = v;
  });
  __syncthreads();
  copy_out(kb, s_kept, nk, -1, keep);
  if (ao) copy_out(ao, s_out, nk, 0.f, max_len);
  if (tid == 0) len_out[b] = nk;
}

// Longer rows: blocks of 8192 tokens, a launch per digit and one that writes.
// ws per sequence: what is found so far {digit 0, rest, digit 1, rest}, and per
// block its counts above the digits found so far, then every block's histogram
// of each level. Nothing needs to start at zero. Bound by the launches: 131072
// tokens 4.4 + 5.9 + 5.8 us for the digits and 8.2 us for the last digit, ranks
// and writes, of which the weights' 512 KiB are a tenth of a microsecond.
constexpr int kBlockKpt = 8, kBlock = kBlockKpt * kThreads;
struct LongWs {
  int32_t* found;   // [B][4]
  int32_t* above;   // [B][2][blocks]
  int32_t* hist;    // [3][B][blocks][kBins]
  float* weight;    // [B][keep]: the kept weights, where acc_out is acc
  int blocks, B;
};
__device__ __forceinline__ int32_t* hist_of(const LongWs& w, int level, int b, int blk) {
  return w.hist + (((int64_t)level * w.B + b) * w.blocks + blk) * kBins;
}
// The sequence's digit of `level` from its blocks' histograms; thread t also
// gets, in before[0..1], what blocks before `blk` hold in its two bins.
__device__ __forceinline__ void find_in_blocks(const LongWs& w, int level, int b, int blk, int n_blk, int want,
                                               int* scratch, int* found, int (&before)[2]) {
  const int32_t* h = hist_of(w, level, b, 0) + (kBins - 2 - 2 * (int)threadIdx.x);
  int c0 = 0, c1 = 0;
  before[0] = before[1] = 0;
  constexpr int kAhead = 8;          // blocks whose loads are under way together
  for (int i0 = 0; i0 < n_blk; i0 += kAhead) {
    int2 v[kAhead];                  // bins 2046 - 2t, 2047 - 2t
#pragma unroll
    for (int u = 0; u < kAhead; ++u) v[u] = *reinterpret_cast<const int2*>(h + (int64_t)min(i0 + u, n_blk - 1) * kBins);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u;
      c0 += i < n_blk ? v[u].y : 0;
      c1 += i < n_blk ? v[u].x : 0;
      before[0] += i < blk ? v[u].y : 0;
      before[1] += i < blk ? v[u].x : 0;
    }
  }
  find_digit(c0, c1, want, scratch, found);
}

template <int LEVEL>
__global__ void __launch_bounds__(kThreads)
    paged_evict_digit_kernel(const float* __restrict__ acc, int64_t acc_ld, const int32_t* __restrict__ seq_len,
                             int max_len, int keep, int n_sink, int n_recent, LongWs w) {
  __shared__ __align__(16) int hist[kBins * kCopies];
  __shared__ int scratch[kWaves], s_found[2];
  const int b = blockIdx.y, blk = blockIdx.x, tid = threadIdx.x, t0 = blk * kBlock;
  const Row r = row_of(seq_len, b, max_len, keep, n_sink, n_recent);
  if (r.want == 0 || t0 >= r.n) return;
  const int n_blk = (r.n + kBlock - 1) / kBlock;
  const float* a = acc + (int64_t)b * acc_ld;
  float x[kBlockKpt];
  uint32_t k[kBlockKpt];
  load_weights<kBlockKpt>(a, t0, max_len, x);
  keys_of<kBlockKpt>(x, t0, r, k);
  clear_bins(hist);
  uint32_t prefix = 0;
  if (LEVEL > 0) {
    int want = r.want, before[2];
    if (LEVEL > 1) {
      prefix = (uint32_t)w.found[b * 4];
      want = w.found[b * 4 + 1];
    }
    find_in_blocks(w, LEVEL - 1, b, blk, n_blk, want, scratch, s_found, before);
    if (blk == 0 && tid < 2) w.found[b * 4 + (LEVEL - 1) * 2 + tid] = s_found[tid];
    // this block's tokens above the digit just found, among those equal before it
    int above = 0;
    constexpr int up = LEVEL == 1 ? 21 : 10;
#pragma unroll
    for (int j = 0; j < kBlockKpt; ++j) {
      const uint32_t d = k[j] >> up;
      const bool in = (LEVEL == 1 || (d >> 11) == prefix) && (d & (kBins - 1)) > (uint32_t)s_found[0];
      above += (int)__popcll(__ballot(in));
    }
    int unused;
    above = waves_sum(above, scratch, &unused);
    if (tid == 0) w.above[((int64_t)b * 2 + LEVEL - 1) * w.blocks + blk] = above;
    prefix = (prefix << 11) | (uint32_t)s_found[0];
  }
  __syncthreads();
  constexpr int shift = LEVEL == 0 ? 21 : LEVEL == 1 ? 10 : 0, width = LEVEL == 2 ? 10 : 11;
  count_digits<kBlockKpt>(k, LEVEL == 0, prefix, shift, width, hist);
  __syncthreads();
  int32_t* h = hist_of(w, LEVEL, b, blk);
  h[tid] = bin_count(hist, tid);
  h[tid + kThreads] = bin_count(hist, tid + kThreads);
}

__global__ void __launch_bounds__(kThreads)
    paged_evict_pick_kernel(const float* __restrict__ acc, int64_t acc_ld, const int32_t* __restrict__ seq_len,
                            int max_len, int keep, int n_sink, int n_recent, int32_t* __restrict__ kept,
                            float* __restrict__ weight, int64_t weight_ld, int ends, int32_t* __restrict__ len_out,
                            LongWs w) {
  __shared__ int scratch[kWaves], s_found[2];
  __shared__ __align__(8) int s_cnt[kWaves][2];
  __shared__ int s_tie0;
  const int b = blockIdx.y, blk = blockIdx.x, tid = threadIdx.x, t0 = blk * kBlock;
  const Row r = row_of(seq_len, b, max_len, keep, n_sink, n_recent);
  int32_t* kb = kept + (int64_t)b * keep;
  const int nk = min(r.n, keep);
  for (int j = max(nk, t0) + tid; j < min(keep, t0 + kBlock); j += kThreads) kb[j] = -1;
  if (ends) {   // the outputs are not the inputs: what follows the kept weights, and the length
    if (weight)
      for (int j = max(nk, t0) + tid; j < min(max_len, t0 + kBlock); j += kThreads) weight[(int64_t)b * weight_ld + j] = 0.f;
    if (blk == 0 && tid == 0) len_out[b] = nk;
  }
  if (t0 >= r.n) return;
  const float* a = acc + (int64_t)b * acc_ld;
  float x[kBlockKpt];
  uint32_t k[kBlockKpt];
  load_weights<kBlockKpt>(a, t0, max_len, x);
  keys_of<kBlockKpt>(x, t0, r, k);
  uint32_t thr = 0xffffffffu;
  int ties = 0, ties0 = 0, at0 = r.lo;
  if (r.want > 0) {
    const int n_blk = (r.n + kBlock - 1) / kBlock;
    int before[2];
    const int d0 = w.found[b * 4], d1 = w.found[b * 4 + 2], want = w.found[b * 4 + 3];
    find_in_blocks(w, 2, b, blk, n_blk, want, scratch, s_found, before);
    const int d2 = s_found[0], bin0 = kBins - 1 - 2 * tid;
    thr = ((uint32_t)d0 << 21) | ((uint32_t)d1 << 10) | (uint32_t)d2;
    ties = s_found[1];
    if (bin0 == d2) s_tie0 = before[0];
    if (bin0 - 1 == d2) s_tie0 = before[1];
    int above = (bin0 > d2 ? before[0] : 0) + (bin0 - 1 > d2 ? before[1] : 0);
    for (int i = tid; i < blk; i += kThreads)
      above += w.above[(int64_t)b * 2 * w.blocks + i] + w.above[((int64_t)b * 2 + 1) * w.blocks + i];
    int unused;
    above = waves_sum(last_lane(lanes_scan(above)), scratch, &unused);   // its barrier publishes s_tie0
    ties0 = s_tie0;
    at0 += above + min(ties, ties0);
  }
  float* wb = weight ? weight + (int64_t)b * weight_ld : nullptr;
  place_kept<kBlockKpt>(a, x, k, r, t0, thr, ties, ties0, at0, nk, s_cnt, [&](int place, int t, float v) {
    if (place < keep) {
      kb[place] = t;
      if (wb) wb[place] = v;
    }
  });
}

// What has to wait until every block has read acc and seq_len, where an output
// is one of them: the weights (if acc_out is acc), the zeros behind them, the
// lengths. grid (blocks, B).
__global__ void __launch_bounds__(kThreads)
    paged_evict_end_kernel(const int32_t* __restrict__ seq_len, int max_len, int keep, float* __restrict__ acc_out,
                           int64_t acc_ld, const float* __restrict__ weight, int64_t weight_ld) {
  const int b = blockIdx.y, nk = min(min(max(seq_len[b], 0), max_len), keep);
  float* ao = acc_out + (int64_t)b * acc_ld;
  for (int j = blockIdx.x * kThreads + threadIdx.x; j < max_len; j += gridDim.x * kThreads) {
    if (j >= nk) ao[j] = 0.f;
    else if (weight) ao[j] = weight[b * weight_ld + j];
  }
}
__global__ void __launch_bounds__(256)
    paged_evict_len_kernel(const int32_t* seq_len, int B, int max_len, int keep, int32_t* len_out) {
  const int b = blockIdx.x * 256 + threadIdx.x;
  if (b < B) len_out[b] = min(min(max(seq_len[b], 0), max_len), keep);
}

// Rows of kept tokens to the pages of another table. grid (ceil(keep / 64),
// B), 256 threads: 64 rows' slots, then their 16-byte pieces, kMovePieces of a
// thread's loads under way at a time. ROW16: pieces per row (0: row16). Bound
// by the rows read and written: 32 x 8192 rows of 1152 bytes 107-123 us, 4.9 to
// 5.6 TB/s (with row16 in place of the constant 7 us more).
constexpr int kMoveRows = 64, kMovePieces = 6;
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
template <int ROW16>
__global__ void __launch_bounds__(256)
    paged_move_kernel(u32x4_t* __restrict__ pool, int row16, Pages src, Pages dst, const int32_t* __restrict__ kept,
                      int keep) {
  __shared__ int s_src[kMoveRows], s_dst[kMoveRows];
  const int b = blockIdx.y, j0 = blockIdx.x * kMoveRows, n16 = ROW16 ? ROW16 : row16;
  if (threadIdx.x < kMoveRows) {
    const int j = j0 + threadIdx.x, t = j < keep ? kept[(int64_t)b * keep + j] : -1;
    int s = -1, d = -1;
    if (t >= 0) {
      s = slot_of(src, src.table + (int64_t)b * src.ld, t);
      d = slot_of(dst, dst.table + (int64_t)b * dst.ld, j);
    }
    s_src[threadIdx.x] = d < 0 ? -1 : s;
    s_dst[threadIdx.x] = d;
  }
  __syncthreads();
  const int total = kMoveRows * n16;
  for (int p0 = threadIdx.x; p0 < total; p0 += 256 * kMovePieces) {
    u32x4_t v[kMovePieces];
    int64_t to[kMovePieces];
#pragma unroll
    for (int u = 0; u < kMovePieces; ++u) {
      // rows that do not move read slot 0, so that every load goes out at once
      const int p = min(p0 + u * 256, total - 1), rw = p / n16, c = p - rw * n16;
      const int s = s_src[rw];
      to[u] = s < 0 || p0 + u * 256 >= total ? -1 : (int64_t)s_dst[rw] * n16 + c;
      v[u] = pool[(int64_t)max(s, 0) * n16 + c];
    }
#pragma unroll
    for (int u = 0; u < kMovePieces; ++u)
      if (to[u] >= 0) pool[to[u]] = v[u];
  }
}

// The same within one table. A kept token's place is never behind it, so a
// batch of rows may be written once all of it is read; the rows that later
// batches read lie behind every place of this one. One workgroup carries a
// 128-byte column of its sequence's rows, kWithin rows a thread under way at a
// time (their entries, then the rows, without a branch between), and all columns
// of a sequence run on one XCD: lines that its columns share, and writes to
// them, meet in one cache: grid (8 x columns, ceil(B / 8)), whose workgroups go
// to the XCDs in turn. 32 x 8192 rows of 1152 bytes 143 us, bound by the
// rows (to other pages 128 us); one sequence of 8192 rows 38 us, bound by the
// waits of its batches. (64-byte columns spread over the XCDs, a row a thread
// and batch: 198 and 40 us; 512 threads 144 and 44 us.)
constexpr int kWithin = 4, kWithinThreads = 1024, kWithinCol = 8;   // pieces a thread and batch; threads; pieces a column
__global__ void __launch_bounds__(kWithinThreads)
    paged_move_within_kernel(u32x4_t* __restrict__ pool, int row16, Pages pg, const int32_t* __restrict__ kept, int keep,
                             int most, int B) {
  const int b = blockIdx.y * 8 + (blockIdx.x & 7);
  const int c = (int)(blockIdx.x >> 3) * kWithinCol + (int)threadIdx.x % kWithinCol;
  if (b >= B) return;
  const int32_t* row = pg.table + (int64_t)b * pg.ld;
  const int32_t* kb = kept + (int64_t)b * keep;
  const int last = (int)min(pg.ld - 1, (int64_t)INT32_MAX);
  constexpr int kRound = kWithinThreads / kWithinCol;
  for (int j0 = 0; j0 < most; j0 += kRound * kWithin) {   // most = min(keep, max_len) places can be taken
    u32x4_t v[kWithin];
    int t[kWithin], ps[kWithin], pd[kWithin], to[kWithin];
#pragma unroll
    for (int u = 0; u < kWithin; ++u) t[u] = kb[min(j0 + u * kRound + (int)threadIdx.x / kWithinCol, keep - 1)];
#pragma unroll
    for (int u = 0; u < kWithin; ++u) {
      const int j = j0 + u * kRound + (int)threadIdx.x / kWithinCol;
      ps[u] = row[min((int)page_index(pg, max(t[u], 0)), last)];
      pd[u] = row[min((int)page_index(pg, j), last)];
    }
#pragma unroll
    for (int u = 0; u < kWithin; ++u) {
      const int j = j0 + u * kRound + (int)threadIdx.x / kWithinCol, tt = max(t[u], 0);
      const int is = (int)page_index(pg, tt), id = (int)page_index(pg, j);
      const int s = is <= last ? slot_in(pg, ps[u], tt - is * pg.size) : -1;
      const int d = id <= last ? slot_in(pg, pd[u], j - id * pg.size) : -1;
      const bool moves = j < keep && t[u] > j && c < row16 && s >= 0;
      to[u] = moves ? d : -1;
      v[u] = pool[(int64_t)(moves ? s : 0) * row16 + (moves ? c : 0)];   // what does not move reads the pool's first piece
    }
    __builtin_amdgcn_s_waitcnt(0x70 | 0xF00);   // vmcnt(0)
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kWithin; ++u)
      if (to[u] >= 0) pool[(int64_t)to[u] * row16 + c] = v[u];
  }
}

// ------------------------------------------------------------------ accepted drafts
// A workgroup per sequence, a thread per 16-byte column. A kept row's place is
// never behind it, and a thread carries its column of all rows, in order: it
// reads kAccept rows before it writes their places, which no later row comes
// from, so nothing waits but for its own loads: the rows' numbers, then their
// entries, then the rows, without a branch between. Bound by these waits: one
// sequence 3.0 us, 256 with four rows each to move 6.9.
constexpr int kAccept = 8;
__global__ void __launch_bounds__(256)
    paged_accept_kernel(u32x4_t* __restrict__ pool, int row16, Pages pg, const int32_t* __restrict__ row0,
                        const int32_t* seq_len, int max_rows, int max_len, const int32_t* __restrict__ kept, int most,
                        const int32_t* __restrict__ n_kept, int32_t* len_out) {   // len_out may be seq_len
  const int b = blockIdx.x;
  const int32_t* kb = kept + (int64_t)b * most;
  const int32_t* row = pg.table + (int64_t)b * pg.ld;
  const int last = (int)min(pg.ld - 1, (int64_t)INT32_MAX);
  int from[kAccept];
#pragma unroll
  for (int u = 0; u < kAccept; ++u) from[u] = kb[min(u, most - 1)];   // asked for beside what says how many there are
  const SeqRows sr = seq_rows(row0, seq_len, pg, b, INT32_MAX, max_rows, max_len);
  const int count = min(min(max(n_kept[b], 0), most), sr.n);
  for (int j0 = 0; j0 < count; j0 += kAccept) {
    int ps[kAccept], pd[kAccept], is[kAccept], id[kAccept];
    if (j0 > 0) {
#pragma unroll
      for (int u = 0; u < kAccept; ++u) from[u] = kb[min(j0 + u, most - 1)];
    }
#pragma unroll
    for (int u = 0; u < kAccept; ++u) {
      const int j = j0 + u;
      // in its place already, or none of the step's: no move
      if (!(j < count && from[u] > j && from[u] < sr.n && sr.pos0 + j >= 0)) from[u] = -1;
      is[u] = (int)page_index(pg, max(sr.pos0 + max(from[u], 0), 0));
      id[u] = (int)page_index(pg, max(sr.pos0 + j, 0));
      ps[u] = row[min(is[u], last)];
      pd[u] = row[min(id[u], last)];
    }
#pragma unroll
    for (int u = 0; u < kAccept; ++u) {
      const int s = is[u] <= last ? slot_in(pg, ps[u], sr.pos0 + from[u] - is[u] * pg.size) : -1;
      const int d = id[u] <= last ? slot_in(pg, pd[u], sr.pos0 + j0 + u - id[u] * pg.size) : -1;
      const bool moves = from[u] >= 0 && s >= 0 && d >= 0;
      ps[u] = moves ? s : -1;
      pd[u] = moves ? d : -1;
    }
    for (int c = threadIdx.x; c < row16; c += blockDim.x) {
      u32x4_t v[kAccept];
#pragma unroll
      for (int u = 0; u < kAccept; ++u)
        if (ps[u] >= 0) v[u] = pool[(int64_t)ps[u] * row16 + c];     // uniform
#pragma unroll
      for (int u = 0; u < kAccept; ++u)
        if (pd[u] >= 0) pool[(int64_t)pd[u] * row16 + c] = v[u];
    }
  }
  __syncthreads();                                         // every thread has read the length
  if (threadIdx.x == 0) len_out[b] = max(sr.pos0 + count, 0);
}

// ------------------------------------------------------------------ copied pages
// The copies' pieces of 16 bytes one after another, kCopyEach * 256 a workgroup;
// a piece's page by the workgroup's first one, which 64 bits name, and a
// division in 32. Bound by the rows: 131072 of 1152 bytes 62.6 us (4.82 TB/s of
// reads and writes; 66.4 with loads and stores that stay in the caches); 12 pages
// by the waits for the page's number and the row, 3.8 us.
constexpr int kCopyEach = 4, kCopyX = 1 << 22;
__global__ void __launch_bounds__(256)
    paged_copy_kernel(u32x4_t* __restrict__ pool, int row16, uint32_t n_slots, int page_size, uint32_t n_pages,
                      const int32_t* __restrict__ src, const int32_t* __restrict__ dst, const int32_t* __restrict__ rows, int n,
                      int64_t page16) {
  const int64_t first = ((int64_t)blockIdx.y * kCopyX + blockIdx.x) * (256 * kCopyEach);
  const int64_t p0 = first / page16;
  const uint32_t in0 = (uint32_t)(first - p0 * page16);    // < page16 < 2^31
  u32x4_t v[kCopyEach];
  int64_t to[kCopyEach];
#pragma unroll
  for (int u = 0; u < kCopyEach; ++u) {
    uint32_t in = in0 + u * 256 + threadIdx.x;
    int64_t p = p0;
    if (in >= (uint32_t)page16) {
      const uint32_t more = in / (uint32_t)page16;
      p += more;
      in -= more * (uint32_t)page16;
    }
    to[u] = -1;
    if (p < n) {
      const uint32_t a = (uint32_t)src[p], d = (uint32_t)dst[p], off = in / (uint32_t)row16;
      const uint32_t limit = rows ? (uint32_t)max(rows[p], 0) : (uint32_t)page_size;
      if (a < n_pages && d < n_pages && off < limit && a * (uint32_t)page_size + off < n_slots &&
          d * (uint32_t)page_size + off < n_slots) {
        v[u] = __builtin_nontemporal_load(pool + (int64_t)a * page16 + in);
        to[u] = (int64_t)d * page16 + in;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kCopyEach; ++u)
    if (to[u] >= 0) __builtin_nontemporal_store(v[u], pool + to[u]);
}

}  // namespace

extern "C" int ech_paged_append(void* pool, int64_t n_slots, int64_t row_bytes, int page_size,
                                const int32_t* page_table, int64_t pt_ld, const int32_t* row0, const int32_t* seq_len,
                                int B, int T, const void* rows, int64_t row_stride, int32_t* status, void* stream) {
  if (!pool || !row0 || !seq_len || (T > 0 && !rows)) return ECH_EINVAL;
  if (B < 1 || B > 65535 || T < 0 || T > (1 << 30) || !pages_ok(n_slots, page_size, page_table, pt_ld)) return ECH_EINVAL;
  if (row_bytes < 16 || row_bytes % 16 || row_bytes > (1 << 20) || row_stride < row_bytes || row_stride % 16 ||
      !aligned16_(pool) || !aligned16_(rows))
    return ECH_EINVAL;
  if (T == 0) return ECH_OK;
  const Pages pg = make_pages(page_table, pt_ld, n_slots, page_size);
  const int wgs = (T + 3) / 4;
  hipLaunchKernelGGL(paged_append_kernel, dim3(std::min(wgs, kAppendX), (wgs + kAppendX - 1) / kAppendX), dim3(256), 0,
                     reinterpret_cast<hipStream_t>(stream),
                     static_cast<uint4*>(pool), (int)(row_bytes / 16), pg, row0, seq_len, B, T,
                     static_cast<const uint4*>(rows), row_stride / 16, status);
  ECH_LAUNCH_CHECK();
  return ECH_OK;
}

// Rows of at most 16384 tokens are one workgroup's work.
constexpr int kRowMost = 16 * kThreads;

static LongWs long_ws(char* ws, int B, int max_len, int keep, size_t* bytes) {
  LongWs w{};
  if (max_len <= kRowMost) {
    *bytes = 0;
    return w;
  }
  auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
  w.B = B;
  w.blocks = (max_len + kBlock - 1) / kBlock;
  const size_t above = up((size_t)B * 4 * 4), hist = above + up((size_t)B * 2 * w.blocks * 4),
               weight = hist + (size_t)3 * B * w.blocks * kBins * 4;
  if (ws) {
    w.found = reinterpret_cast<int32_t*>(ws);
    w.above = reinterpret_cast<int32_t*>(ws + above);
    w.hist = reinterpret_cast<int32_t*>(ws + hist);
    w.weight = reinterpret_cast<float*>(ws + weight);
  }
  *bytes = weight + up((size_t)B * std::min(keep, max_len) * 4);
  return w;
}

static bool evict_shape_ok(int B, int max_len, int keep) {
  return B >= 1 && B <= 65535 && max_len >= 0 && max_len <= (1 << 24) && keep >= 1 && keep <= (1 << 30);
}

extern "C" size_t ech_paged_evict_ws_bytes(int B, int max_len, int keep) {
  if (!evict_shape_ok(B, max_len, keep)) return 0;
  size_t n;
  (void)long_ws(nullptr, B, max_len, keep, &n);
  return n;
}

extern "C" int ech_paged_evict(const float* acc, int64_t acc_ld, const int32_t* seq_len, int B, int max_len, int keep,
                               int n_sink, int n_recent, int32_t* kept, float* acc_out, int32_t* len_out, void* pool,
                               int64_t n_slots, int64_t row_bytes, int page_size, const int32_t* src_table,
                               const int32_t* dst_table, int64_t pt_ld, void* ws, size_t ws_bytes, void* stream) {
  if (!acc || !seq_len || !kept || !len_out) return ECH_EINVAL;
  if (!evict_shape_ok(B, max_len, keep) || acc_ld < max_len || n_sink < 0 || n_recent < 0 ||
      (int64_t)n_sink + n_recent > keep)
    return ECH_EINVAL;
  if (pool) {
    if (!dst_table || !pages_ok(n_slots, page_size, src_table, pt_ld) || row_bytes < 16 || row_bytes % 16 ||
        row_bytes > (1 << 20) || !aligned16_(pool))
      return ECH_EINVAL;
  }
  const size_t need = ech_paged_evict_ws_bytes(B, max_len, keep);
  if (ws_bytes < need || (need && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u)))) return ECH_EINVAL;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
#define ECH_EVICT_ROW(K)                                                                                             \
  hipLaunchKernelGGL(paged_evict_row_kernel<K>, dim3(B), dim3(kThreads), 0, s, acc, acc_ld, seq_len, max_len, keep, \
                     n_sink, n_recent, kept, acc_out, len_out)
  if (max_len <= 4 * kThreads) {
    ECH_EVICT_ROW(4);
  } else if (max_len <= kRowMost) {
    ECH_EVICT_ROW(16);
  } else {
    size_t n;
    const LongWs w = long_ws(static_cast<char*>(ws), B, max_len, keep, &n);
    const dim3 grid(w.blocks, B), block(kThreads);
    hipLaunchKernelGGL(paged_evict_digit_kernel<0>, grid, block, 0, s, acc, acc_ld, seq_len, max_len, keep, n_sink,
                       n_recent, w);
    hipLaunchKernelGGL(paged_evict_digit_kernel<1>, grid, block, 0, s, acc, acc_ld, seq_len, max_len, keep, n_sink,
                       n_recent, w);
    hipLaunchKernelGGL(paged_evict_digit_kernel<2>, grid, block, 0, s, acc, acc_ld, seq_len, max_len, keep, n_sink,
                       n_recent, w);
    ECH_LAUNCH_CHECK();
    const bool same = acc_out == acc || len_out == seq_len, tmp = acc_out == acc;
    const int64_t tmp_ld = std::min(keep, max_len);
    // the blocks past max_len mark unused places where keep is larger
    const dim3 pgrid((std::max(keep, max_len) + kBlock - 1) / kBlock, B);
    hipLaunchKernelGGL(paged_evict_pick_kernel, pgrid, block, 0, s, acc, acc_ld, seq_len, max_len, keep, n_sink, n_recent,
                       kept, tmp ? w.weight : acc_out, tmp ? tmp_ld : acc_ld, (int)!same, len_out, w);
    ECH_LAUNCH_CHECK();
    if (same) {
      if (acc_out) {
        hipLaunchKernelGGL(paged_evict_end_kernel, grid, block, 0, s, seq_len, max_len, keep, acc_out, acc_ld,
                           tmp ? w.weight : nullptr, tmp_ld);
        ECH_LAUNCH_CHECK();
      }
      hipLaunchKernelGGL(paged_evict_len_kernel, dim3((B + 255) / 256), dim3(256), 0, s, seq_len, B, max_len, keep,
                         len_out);
    }
  }
#undef ECH_EVICT_ROW
  ECH_LAUNCH_CHECK();
  if (!pool) return ECH_OK;
  const int row16 = (int)(row_bytes / 16);
  const Pages a = make_pages(src_table, pt_ld, n_slots, page_size), d = make_pages(dst_table, pt_ld, n_slots, page_size);
  const dim3 mgrid((std::min(keep, max_len) + kMoveRows - 1) / kMoveRows, B);
  if (mgrid.x == 0) return ECH_OK;
  if (src_table == dst_table)
    hipLaunchKernelGGL(paged_move_within_kernel, dim3((row16 + kWithinCol - 1) / kWithinCol * 8, (B + 7) / 8),
                       dim3(kWithinThreads), 0, s, static_cast<u32x4_t*>(pool), row16, a, kept, keep, std::min(keep, max_len), B);
  else if (row16 == kPagedChunks)
    hipLaunchKernelGGL(paged_move_kernel<kPagedChunks>, mgrid, dim3(256), 0, s, static_cast<u32x4_t*>(pool), row16, a, d, kept,
                       keep);
  else
    hipLaunchKernelGGL(paged_move_kernel<0>, mgrid, dim3(256), 0, s, static_cast<u32x4_t*>(pool), row16, a, d, kept, keep);
  ECH_LAUNCH_CHECK();
  return ECH_OK;
}

extern "C" int ech_paged_accept(void* pool, int64_t n_slots, int64_t row_bytes, int page_size,
                                const int32_t* page_table, int64_t pt_ld, const int32_t* row0, const int32_t* seq_len,
                                int B, int max_rows, int max_len, const int32_t* kept, int most, const int32_t* n_kept,
                                int32_t* len_out, void* stream) {
  if (!pool || !row0 || !seq_len || !kept || !n_kept || !len_out) return ECH_EINVAL;
  if (!batch_ok(B, 0, max_rows, max_len) || most < 1 || !pages_ok(n_slots, page_size, page_table, pt_ld)) return ECH_EINVAL;
  if (row_bytes < 16 || row_bytes % 16 || row_bytes > (1 << 20) || !aligned16_(pool)) return ECH_EINVAL;
  const Pages pg = make_pages(page_table, pt_ld, n_slots, page_size);
  const int row16 = (int)(row_bytes / 16);
  hipLaunchKernelGGL(paged_accept_kernel, dim3(B), dim3(std::min(256, (row16 + 63) / 64 * 64)), 0,
                     reinterpret_cast<hipStream_t>(stream), static_cast<u32x4_t*>(pool), row16, pg, row0, seq_len, max_rows,
                     max_len, kept, most, n_kept, len_out);
  ECH_LAUNCH_CHECK();
  return ECH_OK;
}

extern "C" int ech_paged_copy(void* pool, int64_t n_slots, int64_t row_bytes, int page_size, const int32_t* src,
                              const int32_t* dst, const int32_t* rows, int n, void* stream) {
  if (!pool || n < 0 || (n > 0 && (!src || !dst))) return ECH_EINVAL;
  if (n_slots < 1 || n_slots >= (1ll << 31) || page_size < 1 || page_size > (1 << 20)) return ECH_EINVAL;
  if (row_bytes < 16 || row_bytes % 16 || row_bytes > (1 << 20) || !aligned16_(pool)) return ECH_EINVAL;
  const int64_t page16 = (int64_t)page_size * (row_bytes / 16);
  const int64_t each = 256 * kCopyEach;
  if (page16 >= (1ll << 31) || page16 * n >= (1ll << 22) * 65535 * each) return ECH_EINVAL;
  if (n == 0) return ECH_OK;
  const int64_t wgs = (page16 * n + each - 1) / each;
  hipLaunchKernelGGL(paged_copy_kernel, dim3((unsigned)std::min<int64_t>(wgs, kCopyX), (unsigned)((wgs + kCopyX - 1) / kCopyX)),
                     dim3(256), 0, reinterpret_cast<hipStream_t>(stream), static_cast<u32x4_t*>(pool), (int)(row_bytes / 16),
                     (uint32_t)n_slots, page_size, (uint32_t)((n_slots + page_size - 1) / page_size), src, dst, rows, n, page16);
  ECH_LAUNCH_CHECK();
  return ECH_OK;
}
