// The attention weight that each cached token received (ech_paged_weight):
//
//   acc_out[b][t] = decay acc_in[b][t] + sum over the step's rows i of b that
//                   see t, and heads h, of exp(scale q[i][h] . k[t] - lse[i][h])
//
// with the lse of ech_paged_attn, so each (row, head) hands out exactly 1. A
// workgroup keeps the keys of 128 tokens in registers (wave w: 32 of them, 144
// registers) and streams the sequence's queries through LDS, 32 at a time; on
// v_mfma_f32_32x32x16_bf16, S[m][token] = Q . K^T leaves a lane one token and
// 16 queries, so the sum over queries stays in the lane and no other lane or
// workgroup adds to a token: the result has one order of additions. Where the
// batch has few token tiles and many queries, the queries are split over
// workgroups and their partial sums joined by a second kernel, in order.
#include <algorithm>

#include "common.hpp"
#include "paged.hpp"

namespace {

typedef __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16 bf16x8_t;
typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16_t;
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kTokWg = 128;                  // tokens per workgroup
constexpr int kQTile = 32;                   // queries per step
constexpr int kKs16 = kPagedRow / 16;
constexpr int kPitchC = 73;
constexpr int kPitch = kPitchC * 16;

// grid (ceil(max_len / 128), B, parts)
__global__ void __launch_bounds__(256, 1)
    paged_weight_kernel(const uint16_t* __restrict__ q, int64_t q_rs, int64_t q_hs, const float* __restrict__ lse,
                        const uint4* __restrict__ pool, Pages pg, const int32_t* __restrict__ row0,
                        const int32_t* __restrict__ seq_len, int T, int H, int max_rows, int max_len, int window,
                        int n_sink, float scale2, const float* __restrict__ acc_in, float* __restrict__ acc_out,
                        int64_t acc_ld, float decay, float* __restrict__ part) {
  __shared__ __align__(16) uint8_t qs[kQTile * kPitch];
  __shared__ float s_lse[kQTile];
  __shared__ int s_pos[kQTile];
  const int b = blockIdx.y, parts = gridDim.z;
  const SeqRows sr = seq_rows(row0, seq_len, pg, b, T, max_rows, max_len);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, col = lane & 31, g = lane >> 5;
  const int tb = blockIdx.x * kTokWg;
  if (tb >= sr.len) return;
  const int t = tb + wave * 32 + col;
  const int slot = t < sr.len ? slot_of(pg, pg.table + (int64_t)b * pg.ld, t) : -1;
  bf16x8_t kf[kKs16];
  {
    const uint4* kp = pool + (int64_t)max(slot, 0) * kPagedChunks + g;
#pragma unroll
    for (int s = 0; s < kKs16; ++s) kf[s] = __builtin_bit_cast(bf16x8_t, kp[2 * s]);
  }
  const int M = sr.n * H, steps = (M + kQTile - 1) / kQTile;
  const int per = (steps + parts - 1) / parts;
  const int s0 = min((int)blockIdx.z * per, steps), s1 = min(s0 + per, steps);
  float w = 0.f;
  for (int i = s0; i < s1; ++i) {
    const int m0 = i * kQTile;
    __syncthreads();
    for (int x = threadIdx.x; x < kQTile * kPagedChunks; x += 256) {
      const int mm = x / kPagedChunks, c = x - mm * kPagedChunks, m = m0 + mm;
      u32x4_t v = {0, 0, 0, 0};
      if (m < M) {
        const int r = m / H, h = m - r * H;
        v = *(reinterpret_cast<const u32x4_t*>(q + (int64_t)(sr.first + r) * q_rs + (int64_t)h * q_hs) + c);
      }
      *reinterpret_cast<u32x4_t*>(qs + mm * kPitch + c * 16) = v;
    }
    if (threadIdx.x < kQTile) {
      const int m = m0 + threadIdx.x;
      s_lse[threadIdx.x] = m < M ? lse[(int64_t)sr.first * H + m] * 1.4426950408889634f : 0.f;
      s_pos[threadIdx.x] = m < M ? sr.pos0 + m / H : -1;
    }
    __syncthreads();
    f32x16_t st;
#pragma unroll
    for (int v = 0; v < 16; ++v) st[v] = 0.f;
    const uint8_t* qr = qs + col * kPitch + g * 16;
#pragma unroll
    for (int s = 0; s < kKs16; ++s)
      st = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t*>(qr + s * 32)), kf[s], st, 0, 0, 0);
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int mm = 8 * (v >> 2) + 4 * g + (v & 3);
      if (sees(s_pos[mm], t, window, n_sink)) w += exp2f(st[v] * scale2 - s_lse[mm]);
    }
  }
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(w), __float_as_uint(w), false, false);
  w = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  if (slot < 0) w = 0.f;
  if (g != 0 || t >= sr.len) return;
  if (parts > 1)
    part[((int64_t)blockIdx.z * gridDim.y + b) * max_len + t] = w;
  else
    acc_out[(int64_t)b * acc_ld + t] = (acc_in ? acc_in[(int64_t)b * acc_ld + t] * decay : 0.f) + w;
}

// grid (ceil(max_len / 256), B)
__global__ void __launch_bounds__(256)
    paged_weight_join_kernel(const float* __restrict__ part, int parts, Pages pg, const int32_t* __restrict__ row0,
                             const int32_t* __restrict__ seq_len, int T, int max_rows, int max_len,
                             const float* __restrict__ acc_in, float* __restrict__ acc_out, int64_t acc_ld, float decay) {
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

int parts_of(int B, int T, int H, int max_rows, int max_len) {
  const int64_t wgs = (int64_t)B * ((max_len + kTokWg - 1) / kTokWg);
  const int64_t steps = ((int64_t)std::min(max_rows, T) * H + kQTile - 1) / kQTile;
  const int64_t want = std::min<int64_t>(256 / std::max<int64_t>(wgs, 1), steps / 8);
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, 64));
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
  const int parts = parts_of(B, T, H, max_rows, max_len);
  const Pages pg = make_pages(page_table, pt_ld, n_slots, page_size);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(paged_weight_kernel, dim3((max_len + kTokWg - 1) / kTokWg, B, parts), dim3(256), 0, s,
                     static_cast<const uint16_t*>(q), q_row_stride, q_head_stride, lse, static_cast<const uint4*>(pool),
                     pg, row0, seq_len, T, H, max_rows, max_len, window, n_sink, sm_scale * 1.4426950408889634f, acc_in,
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
