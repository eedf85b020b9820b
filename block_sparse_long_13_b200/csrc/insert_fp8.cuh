// msa_qknorm_rope_insert_fp8: per-head QK RMSNorm, partial rotary embedding and the insert of the new K and
// V rows into a paged cache of e4m3 codes with one fp32 scale for each (page, KV head).
//
//   q_out[t][h]  = rope(rmsnorm(q[t][h]) * q_norm_w)                              (bf16)
//   y_k[t][g]    = rope(rmsnorm(k_new[t][g]) * k_norm_w),  y_v[t][g] = v_new[t][g]   (fp32, never rounded to bf16)
// and for every (page, g) that the call's rows touch, K and V alike, with a = the largest finite |y| among
// the page's new rows and old = the scale before the call:
//   scale = fit(a)                     if the page begins with one of the call's rows (slot 0 is written)
//         = old                        otherwise, if a <= 448 old
//         = fit(a), and the codes of the page's older rows become e4m3(code * old / scale)  otherwise
//   code[slot] = e4m3(saturate(y / scale)),    fit(a) = the least power of two with 448 fit(a) >= a.
// Rows behind the page's last new row are left as they were.
//
// Two kernels.  kv_insert_fp8_kernel: a CTA owns one (page, head) piece, i.e. up to 128 consecutive rows of one
// sequence inside one block, because the scale needs all of them before any code can be written.  Half a warp
// takes a row's head; the rows stay in registers between the maximum and the rounding, so K and V are read
// once.  The pieces are the first block of each sequence (CTA = sequence) and the blocks that begin inside
// the call's rows (CTA = window of 128 rows, which holds one such block for each sequence that crosses a
// block border in it): num_seqs + total_q / 128 CTAs a head, no search by the host.
// At most 148 CTAs walk the pieces, so that all of them run from the start and q_norm_rope_kernel, which needs nothing
// from them, may be launched beside them (16,384 rows: 166 us behind one another, 106 beside).
// q_norm_rope_kernel: one CTA a row, in and out by bulk copies; bound by HBM.  Both together
// move 5.5 TB/s at 16,384 rows; a single step of 64 rows takes 8.9 us, which two launches and four dependent look-ups set.
//
// Angles: theta^(-2i/r) / 2 pi turns a position, as 64-bit fractions of a turn from a table that the host fills.  Their
// product with the position modulo 2^64 is the fraction of a turn, off by 2^-64 a position (2^-40 at 2^24), in two
// integer multiplications where a double product and its sincos would cost some hundred double instructions; cospi and
// sinpi of it in fp32 lose nothing further.
#pragma once
#include "e4m3.cuh"
#include "launch_order.cuh"
#include "qk_rope_insert.cuh"

namespace msa {

// Threads of a CTA, a row's head to 16 of them, each with ITERS rows in registers.  Sequences of at most 8 rows (a step's
// tokens) take CTAs of 128 threads with one row each: the code is a quarter, four CTAs leave room on an SM, and 64 rows
// take 8.9 us instead of 10.0.  Other calls want a page's 128 rows in one CTA.
constexpr int KVI_THREADS = 512, KVI_ITERS = 4, KVI_GRID = 148;         // of CTAs at most KVI_GRID
constexpr int KVI_FEW_THREADS = 128, KVI_FEW_ROWS = 8, KVI_FEW_GRID = 4 * 148;
static_assert(KVI_THREADS / 16 * KVI_ITERS == 128 && KVI_FEW_THREADS / 16 == KVI_FEW_ROWS, "rows of a CTA");

struct RopeTable { unsigned long long turns[QKR_D / 2]; };   // theta^(-2i/r) / (2 pi) modulo 1, times 2^64, i < rotary_dim / 2

struct KvInsertArgs {
  const __nv_bfloat16* k_new;    // [total_q][Hkv][128]
  const __nv_bfloat16* v_new;
  const __nv_bfloat16* k_w;      // [128]
  uint8_t* k_cache;              // [pages][Hkv][128][128] codes
  uint8_t* v_cache;
  float* k_scale;                // [pages][Hkv]
  float* v_scale;
  const int32_t* q_start;
  const int32_t* ctx_len;
  const int32_t* page_table;
  int num_seqs, total_q, Hkv, max_blocks, num_pages, rotary_dim, pieces, max_q;
  float eps;
};

// cos and sin of the angle of a pair at position p
__device__ __forceinline__ void rope_angle(unsigned long long turns, int p, float& cs, float& sn) {
  const unsigned long long a = turns * static_cast<unsigned long long>(static_cast<long long>(p));
  sincospif(static_cast<float>(static_cast<int>(a >> 32)) * 0x1p-31f, &sn, &cs);   // half turns in [-1, 1]
}

__device__ __forceinline__ float finite_abs(float x) {   // |x|, 0 for infinities and NaN
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}

// Codes of the older rows of a page after its scale grew: e4m3(code * ratio).
template <int THREADS>
__device__ __forceinline__ void rescale_codes(uint8_t* tile, int rows, float ratio) {
  for (int i = threadIdx.x; i < rows * 8; i += THREADS) {
    uint4* p = reinterpret_cast<uint4*>(tile) + i;
    uint4 w = *p;
    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[4];
      e4m3x4_value(u[j], x);
      u[j] = e4m3x4_of(x[0] * ratio, x[1] * ratio, x[2] * ratio, x[3] * ratio);
    }
    *p = w;
  }
}

// e4m3(y / s) of eight numbers, for scales that are no power of two: out of line, so that its divisions do not stand eight
// times in the code that every call runs through.
__device__ __noinline__ uint2 divided_codes(float4 x, float4 y, float s) {
  return make_uint2(e4m3x4_of(__fdiv_rn(x.x, s), __fdiv_rn(x.y, s), __fdiv_rn(x.z, s), __fdiv_rn(x.w, s)),
                    e4m3x4_of(__fdiv_rn(y.x, s), __fdiv_rn(y.y, s), __fdiv_rn(y.z, s), __fdiv_rn(y.w, s)));
}

// One piece: rows t0 .. t0 + n - 1 at positions p0 .. of one block, KV head g, page `page` (valid).
template <int THREADS, int ITERS>
__device__ __forceinline__ void kv_insert_piece(const KvInsertArgs& a, const RopeTable& tab, int t0, int p0, int n, int page,
                                                int g, float (&s_max)[2][THREADS / 32]) {
  constexpr int ROWS = THREADS / 16;                     // at a time
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hl = lane & 15;
  const int row0 = warp * 2 + (lane >> 4);
  const int slot0 = p0 & 127;
  const long tile = static_cast<long>(page) * a.Hkv + g;
  const float k_old = a.k_scale[tile], v_old = a.v_scale[tile];

  // this lane's quads of a K row: a rotation pair (qa, qa + r/8) or two pass-through quads; of a V row: 8 dims
  const int P = a.rotary_dim >> 3;
  const bool rot = hl < P;
  const int qa = rot ? hl : 2 * P + 2 * (hl - P);
  const int ca = 4 * qa, cb = 4 * (rot ? hl + P : qa + 1);

  uint2 ka[ITERS], kb[ITERS];
  uint4 vv[ITERS];
#pragma unroll
  for (int it = 0; it < ITERS; ++it) {
    const int r = it * ROWS + row0;
    ka[it] = kb[it] = make_uint2(0u, 0u);
    vv[it] = make_uint4(0u, 0u, 0u, 0u);
    if (r < n) {
      const long at = (static_cast<long>(t0 + r) * a.Hkv + g) * QKR_D;
      ka[it] = __ldg(reinterpret_cast<const uint2*>(a.k_new + at + ca));
      kb[it] = __ldg(reinterpret_cast<const uint2*>(a.k_new + at + cb));
      vv[it] = __ldg(reinterpret_cast<const uint4*>(a.v_new + at) + hl);
    }
  }
  float wa[4], wb[4];
  load_bf16x4(a.k_w + ca, wa);
  load_bf16x4(a.k_w + cb, wb);
  unsigned long long turns[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) turns[u] = rot ? tab.turns[ca + u] : 0ull;

  float ky[ITERS][8];
  float kmax = 0.f, vmax = 0.f;
#pragma unroll
  for (int it = 0; it < ITERS; ++it) {
    if (it * ROWS >= n) break;                             // uniform
    float xa[4] = {bf16lo(ka[it].x), bf16hi(ka[it].x), bf16lo(ka[it].y), bf16hi(ka[it].y)};
    float xb[4] = {bf16lo(kb[it].x), bf16hi(kb[it].x), bf16lo(kb[it].y), bf16hi(kb[it].y)};
    float ss = 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u) ss += xa[u] * xa[u] + xb[u] * xb[u];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    const float inv = rsqrtf(ss * (1.f / QKR_D) + a.eps);
    const int p = p0 + it * ROWS + row0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float ya = xa[u] * inv * wa[u], yb = xb[u] * inv * wb[u];
      float cs = 1.f, sn = 0.f;
      if (rot) rope_angle(turns[u], p, cs, sn);
      ky[it][u] = rot ? ya * cs - yb * sn : ya;
      ky[it][4 + u] = rot ? yb * cs + ya * sn : yb;
    }
    if (it * ROWS + row0 < n) {                            // rows past the piece hold nothing
#pragma unroll
      for (int u = 0; u < 8; ++u) kmax = fmaxf(kmax, finite_abs(ky[it][u]));
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&vv[it]);
#pragma unroll
      for (int u = 0; u < 4; ++u) vmax = fmaxf(vmax, fmaxf(finite_abs(bf16lo(w[u])), finite_abs(bf16hi(w[u]))));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    kmax = fmaxf(kmax, __shfl_xor_sync(0xFFFFFFFFu, kmax, o));
    vmax = fmaxf(vmax, __shfl_xor_sync(0xFFFFFFFFu, vmax, o));
  }
  if (lane == 0) { s_max[0][warp] = kmax; s_max[1][warp] = vmax; }
  __syncthreads();                                       // every thread has read the old scales
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    kmax = fmaxf(kmax, s_max[0][w]);
    vmax = fmaxf(vmax, s_max[1][w]);
  }
  // a scale that is not a positive number holds nothing: it counts as 0
  const bool k_held = k_old > 0.f && k_old < INFINITY, v_held = v_old > 0.f && v_old < INFINITY;
  const bool k_grown = slot0 == 0 || !k_held || kmax > E4M3_MAX * k_old;
  const bool v_grown = slot0 == 0 || !v_held || vmax > E4M3_MAX * v_old;
  const float ks = k_grown ? e4m3_block_scale(kmax) : k_old, vs = v_grown ? e4m3_block_scale(vmax) : v_old;
  // a power of two's reciprocal is exact, and so is a product with it; other scales (a cache that something else wrote),
  // and 2^127, whose reciprocal is no normal number, are divided by
  const bool exact = (((__float_as_uint(ks) | __float_as_uint(vs)) & 0x7FFFFFu) == 0u) && fminf(ks, vs) >= 0x1p-126f &&
                     fmaxf(ks, vs) <= 0x1p126f;
  const float ki = __uint_as_float(0x7F000000u - __float_as_uint(ks)), vi = __uint_as_float(0x7F000000u - __float_as_uint(vs));
  uint8_t* kt = a.k_cache + tile * (128 * QKR_D);
  uint8_t* vt = a.v_cache + tile * (128 * QKR_D);
#pragma unroll
  for (int it = 0; it < ITERS; ++it) {
    const int r = it * ROWS + row0;
    if (r >= n) break;
    uint8_t* kr = kt + (slot0 + r) * QKR_D;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&vv[it]);
    float z[8];
#pragma unroll
    for (int u = 0; u < 4; ++u) { z[2 * u] = bf16lo(w[u]); z[2 * u + 1] = bf16hi(w[u]); }
    uint2 kc, vc;
    if (exact) {
      const float* y = ky[it];
      kc = make_uint2(e4m3x4_of(y[0] * ki, y[1] * ki, y[2] * ki, y[3] * ki), e4m3x4_of(y[4] * ki, y[5] * ki, y[6] * ki, y[7] * ki));
      vc = make_uint2(e4m3x4_of(z[0] * vi, z[1] * vi, z[2] * vi, z[3] * vi), e4m3x4_of(z[4] * vi, z[5] * vi, z[6] * vi, z[7] * vi));
    } else {
      const float* y = ky[it];
      kc = divided_codes(make_float4(y[0], y[1], y[2], y[3]), make_float4(y[4], y[5], y[6], y[7]), ks);
      vc = divided_codes(make_float4(z[0], z[1], z[2], z[3]), make_float4(z[4], z[5], z[6], z[7]), vs);
    }
    *reinterpret_cast<uint32_t*>(kr + ca) = kc.x;
    *reinterpret_cast<uint32_t*>(kr + cb) = kc.y;
    *reinterpret_cast<uint2*>(vt + (slot0 + r) * QKR_D + 8 * hl) = vc;
  }
  if (slot0 > 0 && k_grown) rescale_codes<THREADS>(kt, slot0, k_held ? __fdiv_rn(k_old, ks) : 0.f);
  if (slot0 > 0 && v_grown) rescale_codes<THREADS>(vt, slot0, v_held ? __fdiv_rn(v_old, vs) : 0.f);
  if (tid == 0) {
    if (k_grown) a.k_scale[tile] = ks;
    if (v_grown) a.v_scale[tile] = vs;
  }
}

template <int THREADS, int ITERS>
__global__ void __launch_bounds__(THREADS, ITERS == 1 ? 4 : 1)
kv_insert_fp8_kernel(const KvInsertArgs a, const __grid_constant__ RopeTable tab) {
  __shared__ float s_max[2][THREADS / 32];
  __shared__ int s_t[128], s_p[128], s_s[128], s_cnt[4];
  pdl_launch_dependents();                               // the queries' kernel needs nothing from this one
  // the cache page of sequence s's block b; -1 (and flagged) if there is none
  auto page_of = [&](int s, int b) -> int {
    const int page = b >= 0 && b < a.max_blocks ? __ldg(a.page_table + static_cast<long>(s) * a.max_blocks + b) : -1;
    if (page >= 0 && page < a.num_pages) return page;
    if (threadIdx.x == 0) flag_error(MSA_DEV_BOUNDS);
    return -1;
  };
  // whether rows t0 .. t0 + nq - 1 at positions p0 .. are a sequence of the batch; none of its pieces is written otherwise
  auto fits = [&](int t0, int nq, int p0) { return p0 >= 0 && t0 >= 0 && t0 + nq <= a.total_q && nq <= a.max_q; };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows = min(a.total_q, __ldg(a.q_start + a.num_seqs));
  for (int piece = blockIdx.x; piece < a.pieces; piece += gridDim.x) {
    const int g = piece % a.Hkv, i = piece / a.Hkv;
    if (i < a.num_seqs) {                                // the block that the sequence's first new row falls in
      const int t0 = __ldg(a.q_start + i), nq = __ldg(a.q_start + i + 1) - t0, p0 = __ldg(a.ctx_len + i) - nq;
      if (nq <= 0) continue;
      if (!fits(t0, nq, p0)) {
        if (tid == 0) flag_error(MSA_DEV_BOUNDS);
        continue;
      }
      const int page = page_of(i, p0 >> 7);
      if (page >= 0) kv_insert_piece<THREADS, ITERS>(a, tab, t0, p0, min(nq, 128 - (p0 & 127)), page, g, s_max);
      __syncthreads();                                   // s_max is written again
      continue;
    }
    // the blocks that begin at a row of this window (not their sequence's first row)
    unsigned vote = 0;
    int t = 0, s = 0, p = 0;
    bool lead = false;
    if (tid < 128) {
      t = (i - a.num_seqs) * 128 + tid;
      if (t < rows) {
        s = find_seq(a.q_start, a.num_seqs, t);
        const int end = __ldg(a.q_start + s + 1);
        p = __ldg(a.ctx_len + s) - end + t;
        const int first = __ldg(a.q_start + s);
        lead = t != first && fits(first, end - first, p - (t - first)) && (p & 127) == 0;
      }
      vote = __ballot_sync(0xFFFFFFFFu, lead);
      if (lane == 0) s_cnt[warp] = __popc(vote);
    }
    __syncthreads();
    if (lead) {
      int at = __popc(vote & ((1u << lane) - 1u));
      for (int w = 0; w < warp; ++w) at += s_cnt[w];
      s_t[at] = t; s_p[at] = p; s_s[at] = s;
    }
    __syncthreads();
    const int n_lead = s_cnt[0] + s_cnt[1] + s_cnt[2] + s_cnt[3];
    for (int j = 0; j < n_lead; ++j) {
      const int page = page_of(s_s[j], s_p[j] >> 7);
      if (page >= 0)
        kv_insert_piece<THREADS, ITERS>(a, tab, s_t[j], s_p[j], min(128, min(rows, __ldg(a.q_start + s_s[j] + 1)) - s_t[j]), page, g, s_max);
      __syncthreads();                                   // s_max is written again
    }
    __syncthreads();                                     // and so are the window's lists
  }
}

struct QNormRopeArgs {
  const __nv_bfloat16* q;        // [total_q][Hq][128]
  __nv_bfloat16* q_out;          // the same shape, q itself or disjoint
  const __nv_bfloat16* q_w;      // [128]
  const int32_t* q_start;
  const int32_t* ctx_len;
  int num_seqs, total_q, Hq, rotary_dim;
  float eps;
};

// CTAS of an SM at least: 8 take 32 registers a thread, which 16,384 rows run faster with (106 us instead of 111) and 64 rows
// slower (10.3 instead of 8.9).
constexpr int QNR_MANY = 6 * 148;                      // rows: more than are in flight without the limit
template <int CTAS>
__global__ void __launch_bounds__(QKR_THREADS, CTAS)
q_norm_rope_kernel(const QNormRopeArgs a, const __grid_constant__ RopeTable tab) {
  extern __shared__ __align__(128) uint8_t qnr_dsmem[];
  __nv_bfloat16* xs = reinterpret_cast<__nv_bfloat16*>(qnr_dsmem);   // [Hq][128]
  __shared__ float s_cos[QKR_D / 2], s_sin[QKR_D / 2];
  __shared__ __align__(16) float s_w[QKR_D];
  __shared__ uint64_t s_bar;
  __shared__ volatile int s_abort;
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t bytes = static_cast<uint32_t>(a.Hq) * QKR_D * 2;
  if (tid == 0) {
    s_abort = 0;
    mbar_init(&s_bar, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(&s_bar, bytes);
    bulk_load(xs, a.q + static_cast<long>(t) * a.Hq * QKR_D, bytes, &s_bar);
  }
  const int s = find_seq(a.q_start, a.num_seqs, t);
  const int end = __ldg(a.q_start + s + 1);
  const bool padded = t >= end;                          // a row behind the last sequence: left as it was
  const int p = __ldg(a.ctx_len + s) - end + t;
  if (tid < a.rotary_dim / 2) rope_angle(tab.turns[tid], p, s_cos[tid], s_sin[tid]);
  if (tid < QKR_D) s_w[tid] = __bfloat162float(a.q_w[tid]);
  const int hl = lane & 15, P = a.rotary_dim >> 3;
  const bool rot = hl < P;
  const int qa = rot ? hl : 2 * P + 2 * (hl - P);
  const int ca = 4 * qa, cb = 4 * (rot ? hl + P : qa + 1);
  __syncthreads();
  if (tid == 0 && !mbar_wait(&s_bar, 0, &s_abort)) mbar_wait_drain(&s_bar, 0);
  __syncthreads();
  if (blockIdx.x == gridDim.x - 1 && tid == 0) pdl_wait();   // this kernel ends after the one that it runs beside
  if (s_abort || padded) return;
  float cs[4], sn[4], wa[4], wb[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    cs[u] = rot ? s_cos[ca + u] : 1.f;
    sn[u] = rot ? s_sin[ca + u] : 0.f;
    wa[u] = s_w[ca + u];
    wb[u] = s_w[cb + u];
  }
  for (int j = 2 * warp + (lane >> 4); j < a.Hq; j += QKR_THREADS / 16) {   // Hq is a multiple of 16: uniform
    __nv_bfloat16* row = xs + j * QKR_D;
    float xa[4], xb[4], oa[4], ob[4];
    load_bf16x4(row + ca, xa);
    load_bf16x4(row + cb, xb);
    float ss = 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u) ss += xa[u] * xa[u] + xb[u] * xb[u];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    const float inv = rsqrtf(ss * (1.f / QKR_D) + a.eps);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float ya = xa[u] * inv * wa[u], yb = xb[u] * inv * wb[u];
      oa[u] = rot ? ya * cs[u] - yb * sn[u] : ya;
      ob[u] = rot ? yb * cs[u] + ya * sn[u] : yb;
    }
    store_bf16x4(row + ca, oa);
    store_bf16x4(row + cb, ob);
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    bulk_store(a.q_out + static_cast<long>(t) * a.Hq * QKR_D, xs, bytes);
    bulk_commit();
    bulk_wait_read_all();                              // shared memory stays valid until the copy has read it
  }
}

}  // namespace msa
