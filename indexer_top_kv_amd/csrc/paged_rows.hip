// Rows that join and leave a resident paged cache: ech_paged_append puts a
// step's new rows into their sequences' pages, ech_paged_evict keeps `keep`
// tokens of each sequence and moves their rows together.
#include <algorithm>

#include "common.hpp"
#include "paged.hpp"

namespace {

// grid (ceil(T / 4)), 256 threads: one wave per row.
__global__ void __launch_bounds__(256)
    paged_append_kernel(uint4* __restrict__ pool, int row16, Pages pg, const int32_t* __restrict__ row0,
                        const int32_t* __restrict__ seq_len, int B, int T, const uint4* __restrict__ rows,
                        int64_t row_stride16, int32_t* __restrict__ status) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
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
  const int pos = seq_len[b] - (row0[b + 1] - t);
  const int slot = pos >= 0 ? slot_of(pg, pg.table + (int64_t)b * pg.ld, pos) : -1;
  if (slot < 0) {
    if (status && lane == 0) atomicOr(status, ECH_ST_FULL);
    return;
  }
  for (int i = lane; i < row16; i += 64) pool[(int64_t)slot * row16 + i] = rows[(int64_t)t * row_stride16 + i];
}

// ------------------------------------------------------------------ eviction
// Order of a weight: larger first; NaN above everything, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float x) { return x != x ? 0xffffffffu : ech::ord_key(x); }

// One workgroup per sequence. A sequence of n > keep tokens keeps its first
// n_sink, its last n_recent, and of the tokens between the `want` = keep -
// n_sink - n_recent with the largest weights, ties to the lower index: the
// want-th largest key is found digit by digit (four of 8 bits) from
// histograms in LDS, then one ordered pass writes the kept tokens. acc_out may
// be acc: a kept token's place is never behind it, and a round's weights are
// read before any are written.
__global__ void __launch_bounds__(1024)
    paged_evict_select_kernel(const float* __restrict__ acc, int64_t acc_ld, const int32_t* __restrict__ seq_len,
                              int max_len, int keep, int n_sink, int n_recent, int32_t* __restrict__ kept,
                              float* __restrict__ acc_out, int32_t* __restrict__ len_out) {
  __shared__ int hist[256];
  __shared__ int scratch[16];
  __shared__ int s_digit, s_rest;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int n = min(max(seq_len[b], 0), max_len);
  const float* a = acc + (int64_t)b * acc_ld;
  int32_t* kb = kept + (int64_t)b * keep;
  float* ao = acc_out ? acc_out + (int64_t)b * acc_ld : nullptr;
  const int nk = min(n, keep);
  uint32_t thr = 0;        // tokens between with a key above thr stay,
  int ties = 0;            // and the first `ties` of those equal to it
  const int lo = n_sink, hi = n - n_recent;
  if (n > keep) {
    int want = keep - n_sink - n_recent;
    uint32_t prefix = 0;
    if (want == 0) {
      thr = 0xffffffffu;
    } else {
      for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int t = lo + tid; t < hi; t += 1024) {
          const uint32_t k = weight_key(a[t]);
          if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
          int rest = want, d = 255;
          while (d > 0 && hist[d] < rest) rest -= hist[d--];
          s_digit = d;
          s_rest = rest;
        }
        __syncthreads();
        prefix = (prefix << 8) | (uint32_t)s_digit;
        want = s_rest;
        __syncthreads();
      }
      thr = prefix;
      ties = want;
    }
  }
  int out = 0, seen = 0;   // kept so far, ties seen so far
  for (int t0 = 0; t0 < n; t0 += 1024) {
    const int t = t0 + tid;
    const float x = t < n ? a[t] : 0.f;
    bool take = t < n, tie = false;
    if (n > keep && t < n && t >= lo && t < hi) {
      const uint32_t k = weight_key(x);
      take = k > thr;
      tie = k == thr;
    }
    int tot;
    const int rank = ech::block_excl_scan<1024>(tie ? 1 : 0, scratch, &tot);
    take = take || (tie && seen + rank < ties);
    seen += tot;
    const int at = out + ech::block_excl_scan<1024>(take ? 1 : 0, scratch, &tot);
    out += tot;
    if (take && at < keep) {
      kb[at] = t;
      if (ao) ao[at] = x;
    }
  }
  for (int j = nk + tid; j < keep; j += 1024) kb[j] = -1;
  __syncthreads();
  if (ao)
    for (int j = nk + tid; j < max_len; j += 1024) ao[j] = 0.f;
  if (tid == 0) len_out[b] = nk;
}

// Rows of kept tokens to the pages of another table. grid (ceil(keep / 4), B),
// one wave per row.
__global__ void __launch_bounds__(256)
    paged_move_kernel(uint4* __restrict__ pool, int row16, Pages src, Pages dst, const int32_t* __restrict__ kept,
                      int keep) {
  const int j = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63, b = blockIdx.y;
  if (j >= keep) return;
  const int t = kept[(int64_t)b * keep + j];
  if (t < 0) return;
  const int s = slot_of(src, src.table + (int64_t)b * src.ld, t);
  const int d = slot_of(dst, dst.table + (int64_t)b * dst.ld, j);
  if (s < 0 || d < 0) return;
  for (int i = lane; i < row16; i += 64) pool[(int64_t)d * row16 + i] = pool[(int64_t)s * row16 + i];
}

// The same within one table. A kept token's place is never behind it, so
// ascending rounds are safe as long as a round's rows are read before any is
// written: one workgroup carries a 64-byte column of every row, alone, 256
// rows a round. grid (ceil(row16 / 4), B), 1024 threads.
__global__ void __launch_bounds__(1024)
    paged_move_within_kernel(uint4* __restrict__ pool, int row16, Pages pg, const int32_t* __restrict__ kept, int keep) {
  const int b = blockIdx.y, c = blockIdx.x * 4 + (threadIdx.x & 3);
  const int32_t* row = pg.table + (int64_t)b * pg.ld;
  for (int j0 = 0; j0 < keep; j0 += 256) {
    const int j = j0 + (threadIdx.x >> 2);
    const int t = j < keep ? kept[(int64_t)b * keep + j] : -1;
    int s = -1, d = -1;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t > j && c < row16) {
      s = slot_of(pg, row, t);
      d = slot_of(pg, row, j);
      if (s >= 0 && d >= 0) v = pool[(int64_t)s * row16 + c];
    }
    __syncthreads();
    if (s >= 0 && d >= 0) pool[(int64_t)d * row16 + c] = v;
    __syncthreads();
  }
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
  hipLaunchKernelGGL(paged_append_kernel, dim3((T + 3) / 4), dim3(256), 0, reinterpret_cast<hipStream_t>(stream),
                     static_cast<uint4*>(pool), (int)(row_bytes / 16), pg, row0, seq_len, B, T,
                     static_cast<const uint4*>(rows), row_stride / 16, status);
  ECH_LAUNCH_CHECK();
  return ECH_OK;
}

extern "C" size_t ech_paged_evict_ws_bytes(int B, int max_len, int keep) {
  (void)B;
  (void)max_len;
  (void)keep;
  return 0;
}

extern "C" int ech_paged_evict(const float* acc, int64_t acc_ld, const int32_t* seq_len, int B, int max_len, int keep,
                               int n_sink, int n_recent, int32_t* kept, float* acc_out, int32_t* len_out, void* pool,
                               int64_t n_slots, int64_t row_bytes, int page_size, const int32_t* src_table,
                               const int32_t* dst_table, int64_t pt_ld, void* ws, size_t ws_bytes, void* stream) {
  if (!acc || !seq_len || !kept || !len_out) return ECH_EINVAL;
  if (B < 1 || B > 65535 || max_len < 0 || max_len > (1 << 30) || acc_ld < max_len || keep < 1 || keep > (1 << 30) ||
      n_sink < 0 || n_recent < 0 || (int64_t)n_sink + n_recent > keep)
    return ECH_EINVAL;
  if (pool) {
    if (!dst_table || !pages_ok(n_slots, page_size, src_table, pt_ld) || row_bytes < 16 || row_bytes % 16 ||
        row_bytes > (1 << 20) || !aligned16_(pool))
      return ECH_EINVAL;
  }
  const size_t need = ech_paged_evict_ws_bytes(B, max_len, keep);
  if (ws_bytes < need || (need && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u)))) return ECH_EINVAL;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(paged_evict_select_kernel, dim3(B), dim3(1024), 0, s, acc, acc_ld, seq_len, max_len, keep, n_sink,
                     n_recent, kept, acc_out, len_out);
  ECH_LAUNCH_CHECK();
  if (!pool) return ECH_OK;
  const int row16 = (int)(row_bytes / 16);
  const Pages a = make_pages(src_table, pt_ld, n_slots, page_size), d = make_pages(dst_table, pt_ld, n_slots, page_size);
  if (src_table == dst_table)
    hipLaunchKernelGGL(paged_move_within_kernel, dim3((row16 + 3) / 4, B), dim3(1024), 0, s, static_cast<uint4*>(pool),
                       row16, a, kept, keep);
  else
    hipLaunchKernelGGL(paged_move_kernel, dim3((keep + 3) / 4, B), dim3(256), 0, s, static_cast<uint4*>(pool), row16, a,
                       d, kept, keep);
  ECH_LAUNCH_CHECK();
  return ECH_OK;
}
