// Sparse GQA attention over a paged cache of e4m3 codes, the plain kernel: one CTA per (row, group).
#pragma once
#include "e4m3.cuh"

namespace msa {

struct AttnFp8Args {
  const __nv_bfloat16* q;        // [total_q][Hq][128]
  const uint8_t* k_cache;        // [pages][Hkv][128][128] codes
  const uint8_t* v_cache;
  const float* k_scale;          // [pages][Hkv]
  const float* v_scale;
  const int32_t* block_idx;      // [total_q][Hkv][topk]
  __nv_bfloat16* out;            // [total_q][Hq][128]
  float* lse;                    // [total_q][Hq] or null
  const int32_t* q_start;
  const int32_t* ctx_len;
  const int32_t* page_table;
  int num_seqs, total_q, Hq, Hkv, topk, max_blocks, num_pages;
  float scale_log2;
};

__global__ void __launch_bounds__(128) attn_fp8_plain_kernel(const AttnFp8Args a) {
  __shared__ float s_q[16][128], s_p[16][129], s_alpha[16];
  const int t = blockIdx.x / a.Hkv, g = blockIdx.x % a.Hkv, tid = threadIdx.x;
  const int s = find_seq(a.q_start, a.num_seqs, t);
  const int end = __ldg(a.q_start + s + 1);
  if (t >= end) return;                              // behind the last sequence
  const int p = __ldg(a.ctx_len + s) - end + t;
  for (int h = 0; h < 16; ++h)
    s_q[h][tid] = __bfloat162float(a.q[(static_cast<long>(t) * a.Hq + g * 16 + h) * 128 + tid]) * a.scale_log2;
  __syncthreads();
  const int hh = tid >> 3, j8 = tid & 7;             // 8 threads per head for the statistics
  float M = -1e30f, L = 0.f, acc[16];
  for (int h = 0; h < 16; ++h) acc[h] = 0.f;
  for (int i = 0; i < a.topk; ++i) {
    const int b = __ldg(a.block_idx + (static_cast<long>(t) * a.Hkv + g) * a.topk + i);
    if (b < 0) continue;
    int page = -1;
    if (b < a.max_blocks && b * 128 <= p) page = __ldg(a.page_table + static_cast<long>(s) * a.max_blocks + b);
    if (page < 0 || page >= a.num_pages) { if (tid == 0) flag_error(MSA_DEV_BOUNDS); continue; }
    const int nvis = min(128, p - b * 128 + 1);
    const long tile = static_cast<long>(page) * a.Hkv + g;
    const float ks = __ldg(a.k_scale + tile), vs = __ldg(a.v_scale + tile);
    float x[16];
    for (int h = 0; h < 16; ++h) x[h] = 0.f;
    const uint32_t* k = reinterpret_cast<const uint32_t*>(a.k_cache + (tile * 128 + tid) * 128);
    for (int d = 0; d < 32; ++d) {
      float kv[4];
      e4m3x4_value(__ldg(k + d), kv);
#pragma unroll
      for (int h = 0; h < 16; ++h)
#pragma unroll
        for (int u = 0; u < 4; ++u) x[h] = fmaf(s_q[h][4 * d + u], kv[u], x[h]);
    }
#pragma unroll
    for (int h = 0; h < 16; ++h) s_p[h][tid] = tid < nvis ? x[h] * ks : -INFINITY;
    __syncthreads();
    float m = -1e30f;
    for (int k2 = j8; k2 < 128; k2 += 8) m = fmaxf(m, s_p[hh][k2]);
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float Mn = fmaxf(M, m), al = exp2f(M - Mn);
    float l = 0.f;
    for (int k2 = j8; k2 < 128; k2 += 8) {
      const float e = exp2f(s_p[hh][k2] - Mn);
      s_p[hh][k2] = e;
      l += e;
    }
    for (int o = 4; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    L = L * al + l;
    M = Mn;
    if (j8 == 0) s_alpha[hh] = al;
    __syncthreads();
    float o[16];
#pragma unroll
    for (int h = 0; h < 16; ++h) o[h] = 0.f;
    const uint8_t* v = a.v_cache + tile * 128 * 128 + tid;
    for (int k2 = 0; k2 < nvis; ++k2) {
      const float vv = e4m3x2_value(v[k2 * 128]).x;
#pragma unroll
      for (int h = 0; h < 16; ++h) o[h] = fmaf(s_p[h][k2], vv, o[h]);
    }
#pragma unroll
    for (int h = 0; h < 16; ++h) acc[h] = acc[h] * s_alpha[h] + o[h] * vs;
    __syncthreads();
  }
  __syncthreads();
  if (j8 == 0) {
    s_alpha[hh] = L;
    if (a.lse) a.lse[static_cast<long>(t) * a.Hq + g * 16 + hh] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
  }
  __syncthreads();
  for (int h = 0; h < 16; ++h)
    a.out[(static_cast<long>(t) * a.Hq + g * 16 + h) * 128 + tid] =
        __float2bfloat16_rn(s_alpha[h] == 0.f ? 0.f : acc[h] / s_alpha[h]);
}

}  // namespace msa
