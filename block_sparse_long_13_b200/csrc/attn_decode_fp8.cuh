// msa_attn_decode_fp8: sparse GQA attention for a few queries per sequence over a paged cache of e4m3 codes
// with one fp32 scale for each (page, KV head), on the 5th-generation tensor cores.
//
// For query row t (position p) and KV group g, head h, over the visible keys j of the selected blocks b:
//   x_j = (scale log2 e) ks_b (q_h . ck_j),  out = sum_j 2^(x_j - M) vs_b cv_j / sum_j 2^(x_j - M),
//   lse = (M + log2 sum_j 2^(x_j - M)) ln 2,    ck, cv the codes' values.
//
// The codes go from TMA straight into the tensor cores: both products run as kind::f8f6f4 MMAs in the
// transposed form ("swap AB": a row has only 16 query heads),
//   S^T = K_b Q^T   (M = 128 keys, N = 16 heads, K = 128 dims),   O_b^T = V_b^T P^T   (M = 128 dims, K = 128 keys),
// which want Q and P in 8 bits too.  Neither is rounded to 8 bits: each is the sum of two e4m3 numbers, high and
// low part, multiplied one after the other into the same fp32 accumulator.
//   Q: scaled per head by a power of two so that the largest |q| is in (224, 448].  A bf16 number has 8
//      significant bits; the high part takes 4 of them, and the rest is a multiple of q's last bit by at most 8
//      of them either way, which 4 bits hold: exact, down to elements 2^-11 below the head's largest (below it
//      the error is 2^-10 of a scaled unit, at most 2^-17 of the largest element).
//   P: 256 2^(x - M) <= 256, rounded first to f16 (2^-12 of itself), then high + low: 2^-9 of itself, 2^-18 of the
//      row's largest at least.  That is what bf16 probabilities (2^-9) lose, and the sum of probabilities is
//      taken from the unrounded fp32 values.
// Converting the tiles to 16 bits in shared memory instead would read and write 96 KiB of it a block and
// keep a warpgroup busy; the second MMA of each pair costs 32 KiB of reads by the tensor core.
//
// Bound by HBM: 32 KiB a block and group.  148 persistent CTAs, one per SM; CTA c takes the slots
// [c n / grid, (c + 1) n / grid) of the n = rows x groups x topk slots, so that every CTA streams the same number of
// blocks whatever the batch (whole rows per CTA would leave 64 x 4 groups two rounds over 148 CTAs: 0.86 busy).  A
// (row, group) that a border cuts leaves partial sums, which attn_decode_fp8_merge_kernel joins.
//
// Warps: 0 issues the copies (6 stages of K + V tiles, 192 KiB in flight), 1 the MMAs of S^T, 12 those of O^T, 2 splits
// the queries, 3 looks up slots (32 at a time: block id, sequence, page, scales), 4-7 run the softmax (thread = key; running maxima over
// the row's blocks, so a block's probabilities have the scale of the row so far), 8-11 keep the output (thread =
// dim): acc = acc 2^(M_old - M) + vs_b O_b.  Every wait is bounded.
#pragma once
#include "attn_decode.cuh"
#include "e4m3.cuh"

namespace msa {

constexpr int ATD8_THREADS = 416;
constexpr int ATD8_GRID = 148;         // CTAs at most
constexpr int ATD8_STAGES = 6;         // K + V tiles of a block
constexpr int ATD8_TILE = 16384;       // one K or V block: [128 keys][128 dims] codes, 128-byte swizzle
constexpr int ATD8_RING = 4;           // S^T and O^T accumulators (TMEM), P^T tiles and rescaling factors (shared memory)
constexpr int ATD8_PT = 4096;          // P^T or Q of a row: [high, low][2 KiB]
constexpr int ATD8_BATCHES = 4;        // slot records in flight, 32 each
constexpr int ATD8_SMEM = ATD8_STAGES * 2 * ATD8_TILE + ATD8_RING * ATD8_PT + 2 * ATD8_PT + 1024;
constexpr uint32_t ATD8_TM_S = 0, ATD8_TM_O = ATD8_RING * 32, ATD8_TMEM = 256;   // S^T: 32 columns (high, low part), O^T: 16
constexpr int ATD8_PART = 16 * 128 + 32;   // floats of a partial result: sums [16][128], maxima [16], sums of p [16]
constexpr float ATD8_LOW = -1e30f;     // start of the running maxima (finite: -inf - -inf is NaN)

struct AttnDecodeFp8Args {
  const __nv_bfloat16* q;        // [total_q][Hq][128]
  const float* k_scale;          // [pages][Hkv]
  const float* v_scale;
  const int32_t* block_idx;      // [total_q][Hkv][topk]
  __nv_bfloat16* out;            // [total_q][Hq][128]
  float* lse;                    // [total_q][Hq] or null
  const int32_t* q_start;
  const int32_t* ctx_len;
  const int32_t* page_table;
  float* part;                   // [2 grid][ATD8_PART]: a CTA's first and last cut (row, group)
  int num_seqs, Hq, Hkv, topk, max_blocks, num_pages, n_slots;
  int total_q;
  bool once;                     // tiles are read by one row each
  float scale_log2;
};

__device__ __forceinline__ int atd8_first(int n_slots, int c, int grid) {
  return static_cast<int>(static_cast<long>(n_slots) * c / grid);
}

// kind::f8f6f4 with e4m3 operands, fp32 accumulate
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void umma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// descriptor of an unswizzled MN-major 8-bit operand 16 elements wide: [k][16] bytes, 8-row groups 128 bytes apart
__device__ __forceinline__ uint64_t sdesc_rows16(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(8) << 16) | (static_cast<uint64_t>(8) << 32) |
         (static_cast<uint64_t>(1) << 46);
}

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// two values (<= 448) as high + low e4m3 pairs
__device__ __forceinline__ void e4m3x2_split(float a, float b, uint32_t& hi, uint32_t& lo) {
  uint32_t h2, back, d;
  uint16_t u, v;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h2) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(u) : "r"(h2));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h2), "r"(back));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(v) : "r"(d));
  hi = u;
  lo = v;
}

__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The sequence of row t: the row's share of the sequences first (exact when all have as many rows), then a search.
__device__ __forceinline__ int find_seq_even(const int32_t* q_start, int num_seqs, int total_q, int t) {
  const int s = min(num_seqs - 1, static_cast<int>(static_cast<long>(t) * num_seqs / total_q));
  if (__ldg(q_start + s) <= t && t < __ldg(q_start + s + 1)) return s;
  return find_seq(q_start, num_seqs, t);
}

__global__ void __launch_bounds__(ATD8_THREADS, 1)
attn_decode_fp8_kernel(const __grid_constant__ CUtensorMap tmap_k,    // k codes as [P*Hkv*128][128]
                       const __grid_constant__ CUtensorMap tmap_v, const AttnDecodeFp8Args a) {
  extern __shared__ __align__(1024) uint8_t dsmem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;                                   // stages of [K 16 KiB][V 16 KiB]
  uint8_t* q_s = ring + ATD8_STAGES * 2 * ATD8_TILE;      // 2 x [high, low][16 heads][128] (128-byte swizzle)
  uint8_t* p_s = q_s + 2 * ATD8_PT;                       // ring of [high, low][128 keys][16 heads]

  // Ring slot of block i: s_full S^T is in TMEM; p_full its P^T and factors are in shared memory (and S^T is read);
  // o_full O^T is in TMEM (and P^T is read); o_empty O^T and the factors are read.  So p_full(i - RING) also says
  // that S^T(i) may be written, and o_empty(i - RING), which the softmax waits for, that P^T(i) and O^T(i) may be.
  __shared__ uint64_t k_full[ATD8_STAGES], v_full[ATD8_STAGES], kv_empty[ATD8_STAGES], s_full[ATD8_RING],
      p_full[ATD8_RING], o_full[ATD8_RING], o_empty[ATD8_RING], rec_full[ATD8_BATCHES], rec_empty[ATD8_BATCHES],
      q_full[2], q_empty[2], us_full[2], us_empty[2], drain_bar[2];
  __shared__ __align__(16) int4 s_rec[ATD8_BATCHES * 32]; // slot: TMA row or -1, visible keys, K scale, V scale
  __shared__ uint32_t s_mask[ATD8_BATCHES];               // slots of the batch that hold a block
  __shared__ __align__(16) float s_fq[2][16];             // softmax scale x log2 e / the query's power of two
  __shared__ __align__(16) float s_red[2][4][16];         // per-warp maxima of a block, by block parity
  __shared__ __align__(16) float s_run[4][2][16];         // per warp: the row's running maxima, the block's factors
  __shared__ __align__(16) float s_alpha[ATD8_RING][16];  // 2^(M_old - M) of a block
  __shared__ __align__(16) float s_m[2][16], s_l[2][4][16];   // of a finished (row, group): maxima, per-warp sums of p
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lo = atd8_first(a.n_slots, blockIdx.x, gridDim.x);
  const int n = atd8_first(a.n_slots, blockIdx.x + 1, gridDim.x) - lo;   // > 0: grid <= n_slots
  const int nbatch = (n + 31) >> 5;
  const int unit0 = lo / a.topk;
  const int left0 = a.topk - (lo - unit0 * a.topk);       // slots of the first (row, group) in this range
  if (tid == 0) {
    pdl_launch_dependents();
    s_abort = 0;
    for (int i = 0; i < ATD8_STAGES; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < ATD8_RING; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_empty[i], 4);
    }
    for (int i = 0; i < ATD8_BATCHES; ++i) {
      mbar_init(&rec_full[i], 1);
      mbar_init(&rec_empty[i], 11);                       // producer, two issuers, 4 softmax and 4 output warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 5);                          // issuer, 4 softmax warps
      mbar_init(&us_full[i], 4);
      mbar_init(&us_empty[i], 4);
    }
    mbar_init(&drain_bar[0], 1);
    mbar_init(&drain_bar[1], 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, ATD8_TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // The records of batch bt: lane's slot, and which of the batch's slots hold a block.  Warp-uniform result.
  auto take_batch = [&](int bt, int4& r, uint32_t& mask) -> bool {
    const int rb = bt & (ATD8_BATCHES - 1);
    if (!mbar_wait_warp(&rec_full[rb], (bt / ATD8_BATCHES) & 1, &s_abort)) return false;
    r = s_rec[rb * 32 + lane];
    mask = s_mask[rb];
    __syncwarp();
    if (lane == 0) mbar_arrive(&rec_empty[rb]);
    return true;
  };

  if (warp == 3) {
    // ------------------------------------------------------------ slot records, 32 lookups at a time
    for (int bt = 0; bt < nbatch; ++bt) {
      int4 rec = make_int4(-1, 0, 0, 0);
      const int i = lo + bt * 32 + lane;
      if (bt * 32 + lane < n) {
        const int b = __ldg(a.block_idx + i);
        const int unit = i / a.topk, t = unit / a.Hkv, g = unit - t * a.Hkv;
        const int s = find_seq_even(a.q_start, a.num_seqs, a.total_q, t);
        const int end = __ldg(a.q_start + s + 1);
        if (b >= 0 && t < end) {                          // rows behind the last sequence hold nothing
          const int p = __ldg(a.ctx_len + s) - end + t;
          const int page = b < a.max_blocks && b * 128 <= p ? __ldg(a.page_table + static_cast<long>(s) * a.max_blocks + b) : -1;
          if (page >= 0 && page < a.num_pages) {
            const int tile = page * a.Hkv + g;
            rec = make_int4(tile * 128, min(128, p - b * 128 + 1), __float_as_int(__ldg(a.k_scale + tile)),
                            __float_as_int(__ldg(a.v_scale + tile)));
          } else {
            flag_error(MSA_DEV_BOUNDS);
          }
        }
      }
      const int rb = bt & (ATD8_BATCHES - 1);
      if (!mbar_wait_warp(&rec_empty[rb], ((bt / ATD8_BATCHES) & 1) ^ 1, &s_abort)) break;
      s_rec[rb * 32 + lane] = rec;
      const uint32_t mask = __ballot_sync(0xFFFFFFFFu, rec.x >= 0);
      if (lane == 0) s_mask[rb] = mask;
      __syncwarp();
      if (lane == 0) mbar_arrive(&rec_full[rb]);
    }
  } else if (warp == 0) {
    // ------------------------------------------------------------ copies
    if (lane == 0) {
      tma_prefetch_desc(&tmap_k);
      tma_prefetch_desc(&tmap_v);
    }
    const uint64_t pol = l2_policy_evict_first();
    int st = 0, ph = 1, used = 0;
    bool ok = true;
    for (int bt = 0; bt < nbatch && ok; ++bt) {
      int4 r;
      uint32_t mask;
      if (!take_batch(bt, r, mask)) break;
      for (; mask; mask &= mask - 1) {
        const int row = __shfl_sync(0xFFFFFFFFu, r.x, __ffs(mask) - 1);
        if (!mbar_wait_warp(&kv_empty[st], ph, &s_abort)) { ok = false; break; }
        if (lane == 0) {
          uint8_t* dst = ring + st * 2 * ATD8_TILE;
          mbar_arrive_expect_tx(&k_full[st], ATD8_TILE);
          mbar_arrive_expect_tx(&v_full[st], ATD8_TILE);
          if (a.once) {
            tma_load_2d_hint(dst, &tmap_k, &k_full[st], 0, row, pol);
            tma_load_2d_hint(dst + ATD8_TILE, &tmap_v, &v_full[st], 0, row, pol);
          } else {
            tma_load_2d(dst, &tmap_k, &k_full[st], 0, row);
            tma_load_2d(dst + ATD8_TILE, &tmap_v, &v_full[st], 0, row);
          }
        }
        ++used;
        if (++st == ATD8_STAGES) { st = 0; ph ^= 1; }
      }
    }
    if (lane == 0 && s_abort) {              // let every issued copy land before the CTA exits
      for (int i = 0; i < ATD8_STAGES && i < used; ++i) {
        const int par = ((used - 1 - i) / ATD8_STAGES) & 1;   // of the stage's last use
        mbar_wait_drain(&k_full[i], par);
        mbar_wait_drain(&v_full[i], par);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ S^T = K_b Q^T, one thread
    // Q's high and low part are the two halves of one N = 32 operand: an MMA this narrow takes 47 clocks whatever its
    // N (measured, N <= 64), so one pass over K for both halves the MMAs; the softmax adds the halves.
    if (lane == 0) {
      const uint32_t id_s = idesc_e4m3(128, 32, false, false);   // A = K_b (K-major), B = Q (K-major)
      const uint64_t k_d = sdesc_sw128(smem_u32(ring), 16, 1024);
      const uint64_t q_d = sdesc_sw128(smem_u32(q_s), 16, 1024);
      int st = 0, ph = 0, left = left0, uq = 0;
      uint32_t ns = 0;
      bool ok = true, need_q = true;
      for (int bt = 0; bt < nbatch && ok; ++bt) {
        const int rb = bt & (ATD8_BATCHES - 1);
        if (!mbar_wait(&rec_full[rb], (bt / ATD8_BATCHES) & 1, &s_abort)) break;
        const uint32_t mask = s_mask[rb];
        mbar_arrive(&rec_empty[rb]);
        const int cnt = min(32, n - bt * 32);
        for (int j = 0; j < cnt && ok; ++j) {
          const bool ends = --left == 0 || bt * 32 + j == n - 1;
          if (need_q && (((mask >> j) & 1) || ends)) {
            ok = mbar_wait(&q_full[uq & 1], (uq >> 1) & 1, &s_abort);
            need_q = false;
          }
          if (ok && ((mask >> j) & 1)) {
            const uint32_t ss = ns % ATD8_RING;
            ok = mbar_wait(&k_full[st], ph, &s_abort) &&
                 (ns < ATD8_RING || mbar_wait(&p_full[ss], (ns / ATD8_RING - 1) & 1, &s_abort));
            if (!ok) break;
            tc_fence_after();
            const uint64_t kd = k_d + ((st * 2 * ATD8_TILE) >> 4), qd = q_d + (((uq & 1) * ATD8_PT) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)   // 32 dims per step, within a 128-byte row
              umma_e4m3_ss(tmem + ATD8_TM_S + ss * 32, kd + kk * 2, qd + kk * 2, id_s, kk > 0 ? 1u : 0u);
            umma_commit(&s_full[ss]);
            ++ns;
            if (++st == ATD8_STAGES) { st = 0; ph ^= 1; }
          }
          if (ends && ok) {
            umma_commit(&q_empty[uq & 1]);
            ++uq;
            need_q = true;
            left = a.topk;
          }
        }
      }
      if (s_abort) {
        umma_commit(&drain_bar[0]);
        mbar_wait_drain(&drain_bar[0], 0);
      }
    }
  } else if (warp == 12) {
    // ------------------------------------------------------------ O_b^T = V_b^T P^T, one thread
    if (lane == 0) {
      const uint32_t id_pv = idesc_e4m3(128, 16, true, true);    // A = V_b^T, B = P^T (both MN-major)
      const uint64_t v_d = sdesc_sw128(smem_u32(ring) + ATD8_TILE, ATD8_TILE, 1024);
      const uint64_t p_d = sdesc_rows16(smem_u32(p_s));
      int st = 0, ph = 0;
      uint32_t np = 0;
      bool ok = true;
      for (int bt = 0; bt < nbatch && ok; ++bt) {
        const int rb = bt & (ATD8_BATCHES - 1);
        if (!mbar_wait(&rec_full[rb], (bt / ATD8_BATCHES) & 1, &s_abort)) break;
        const int cnt = __popc(s_mask[rb]);
        mbar_arrive(&rec_empty[rb]);
        for (int j = 0; j < cnt; ++j) {
          const uint32_t ps = np % ATD8_RING;
          ok = mbar_wait(&v_full[st], ph, &s_abort) && mbar_wait(&p_full[ps], (np / ATD8_RING) & 1, &s_abort);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = v_d + ((st * 2 * ATD8_TILE) >> 4), pd = p_d + ((ps * ATD8_PT) >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)     // 32 keys per step: 4 KiB of V rows, 512 bytes of P rows; high, then low part
            umma_e4m3_ss(tmem + ATD8_TM_O + ps * 16, vd + (kk & 3) * 256, pd + (kk >> 2) * 128 + (kk & 3) * 32, id_pv, kk > 0 ? 1u : 0u);
          umma_commit(&o_full[ps]);
          umma_commit(&kv_empty[st]);
          ++np;
          if (++st == ATD8_STAGES) { st = 0; ph ^= 1; }
        }
      }
      if (s_abort) {
        umma_commit(&drain_bar[1]);
        mbar_wait_drain(&drain_bar[1], 0);
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ queries: lane = half a head
    const int nu = (lo + n - 1) / a.topk - unit0 + 1;
    const int h = lane >> 1, half = lane & 1;
    uint4 nxt[8];
    auto load = [&](int unit) {
      const int t = unit / a.Hkv, g = unit - t * a.Hkv;
      const uint4* p = reinterpret_cast<const uint4*>(a.q + (static_cast<long>(t) * a.Hq + g * 16 + h) * 128 + half * 64);
#pragma unroll
      for (int i = 0; i < 8; ++i) nxt[i] = __ldg(p + i);
    };
    load(unit0);
    for (int u = 0; u < nu; ++u) {
      uint4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = nxt[i];
      if (u + 1 < nu) load(unit0 + u + 1);
      uint32_t m2 = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m2 = __vmaxu2(m2, __vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu));
        m2 = __vmaxu2(m2, __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu));
      }
      uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);           // |largest| as bf16 bits (NaN above infinity above the rest)
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      // times 2^k: the largest comes to (224, 448], 448 = 1.75 * 2^8
      const int k = min(120, 135 - static_cast<int>(m >> 7) - ((m & 0x7Fu) > 0x60u ? 1 : 0));
      const float mult = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
      const int qb = u & 1;
      if (!mbar_wait_warp(&q_empty[qb], ((u >> 1) & 1) ^ 1, &s_abort)) break;
      if (half == 0)
        s_fq[qb][h] = m >= 0x7F80u ? __uint_as_float(0x7FC00000u)   // an infinite or NaN query: its head is NaN
                                   : a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
      uint8_t* qt = q_s + qb * ATD8_PT;
#pragma unroll
      for (int i = 0; i < 4; ++i) {                       // 16 dims: 16 bytes of each part
        uint32_t hi[4], lw[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint4& v = x[2 * i + (w >> 1)];
          const uint32_t w0 = (w & 1) ? v.z : v.x, w1 = (w & 1) ? v.w : v.y;
          uint32_t h0, l0, h1, l1;
          e4m3x2_split(bf16lo(w0) * mult, bf16hi(w0) * mult, h0, l0);
          e4m3x2_split(bf16lo(w1) * mult, bf16hi(w1) * mult, h1, l1);
          hi[w] = h0 | (h1 << 16);
          lw[w] = l0 | (l1 << 16);
        }
        const uint32_t at = sw128_offset(h, half * 64 + i * 16);
        *reinterpret_cast<uint4*>(qt + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(qt + 2048 + at) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[qb]);
    }
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ softmax: thread = key
    // The four warps meet at one barrier a block (the exchange of their maxima), which also carries a failed wait
    // to all of them: after a failed wait a warp goes to that barrier and leaves, and so do the others there or at
    // the last barrier, behind the last slot.
    const int sw = warp - 4, row = sw * 32 + lane;
    const uint32_t s_addr = tmem + (static_cast<uint32_t>(sw * 32) << 16) + ATD8_TM_S;
    // Lane h (and h + 16) keeps the running maximum of head h; the sums are per thread, i.e. per key.
    float mine = ATD8_LOW, L[16], fq[16];
#pragma unroll
    for (int h = 0; h < 16; ++h) L[h] = 0.f;
    int st = 0, ph = 0;                      // the block's stage
    uint32_t nb = 0;
    int u = 0, left = left0;
    bool ok = true, left_group = false, need_q = true;
    auto take_q = [&]() -> bool {
      need_q = false;
      if (!mbar_wait_warp(&q_full[u & 1], (u >> 1) & 1, &s_abort)) return false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = *reinterpret_cast<const float4*>(&s_fq[u & 1][4 * i]);
        fq[4 * i] = f.x; fq[4 * i + 1] = f.y; fq[4 * i + 2] = f.z; fq[4 * i + 3] = f.w;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[u & 1]);
      return true;
    };
    for (int bt = 0; bt < nbatch && ok && !left_group; ++bt) {
      int4 r;
      uint32_t mask;
      if (!take_batch(bt, r, mask)) { ok = false; break; }
      const int cnt = min(32, n - bt * 32);
      for (int j = 0; j < cnt; ++j) {
        if ((mask >> j) & 1) {
          const int nvis = __shfl_sync(0xFFFFFFFFu, r.y, j);
          const float ks = __int_as_float(__shfl_sync(0xFFFFFFFFu, r.z, j));
          const uint32_t ss = nb % ATD8_RING, par = (nb / ATD8_RING) & 1;
          if (need_q) ok = take_q();
          ok = ok && mbar_wait_warp(&s_full[ss], par, &s_abort);
          float x[16];
          if (ok) {
            tc_fence_after();
            float v[32];
            tmem_ld32(s_addr + ss * 32, v);
            tmem_ld_wait();
            tc_fence_before();
            float wm[16];
#pragma unroll
            for (int h = 0; h < 16; ++h) {
              x[h] = row < nvis ? (v[h] + v[16 + h]) * (fq[h] * ks) : -INFINITY;
              wm[h] = warp_max(x[h]);
            }
            if (lane == 0) {
              float4* d = reinterpret_cast<float4*>(s_red[nb & 1][sw]);
#pragma unroll
              for (int i = 0; i < 4; ++i) d[i] = make_float4(wm[4 * i], wm[4 * i + 1], wm[4 * i + 2], wm[4 * i + 3]);
            }
            // the P^T tile and the factors of the block RING back are read
            ok = mbar_wait_warp(&o_empty[ss], par ^ 1, &s_abort);
          }
          if (named_bar_any(1, 128, !ok)) { left_group = true; break; }
          // every warp joins the four maxima for itself, a head per lane, and hands them to its lanes
          const float(&red)[4][16] = s_red[nb & 1];
          const int h16 = lane & 15;
          const float bm = fmaxf(fmaxf(red[0][h16], red[1][h16]), fmaxf(red[2][h16], red[3][h16]));
          const float old = mine;
          mine = fmaxf(old, bm);
          const float fac = exp2f(old - mine);
          if (lane < 16) {
            s_run[sw][0][lane] = mine;
            s_run[sw][1][lane] = fac;
            if (sw == 0) s_alpha[ss][lane] = fac;
          }
          const bool grown = __any_sync(0xFFFFFFFFu, mine > old);
          __syncwarp();
          float M[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 m = *reinterpret_cast<const float4*>(&s_run[sw][0][4 * i]);
            M[4 * i] = m.x; M[4 * i + 1] = m.y; M[4 * i + 2] = m.z; M[4 * i + 3] = m.w;
          }
          if (grown) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 f = *reinterpret_cast<const float4*>(&s_run[sw][1][4 * i]);
              L[4 * i] *= f.x; L[4 * i + 1] *= f.y; L[4 * i + 2] *= f.z; L[4 * i + 3] *= f.w;
            }
          }
          uint32_t hi[4], lw[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float p[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              p[v] = exp2f((x[4 * i + v] - M[4 * i + v]) + 8.f);     // 256 2^(x - M); 2^-inf = 0
              L[4 * i + v] += p[v];
            }
            uint32_t h0, l0, h1, l1;
            e4m3x2_split(p[0], p[1], h0, l0);
            e4m3x2_split(p[2], p[3], h1, l1);
            hi[i] = h0 | (h1 << 16);
            lw[i] = l0 | (l1 << 16);
          }
          uint8_t* pt = p_s + ss * ATD8_PT + row * 16;
          *reinterpret_cast<uint4*>(pt) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(pt + 2048) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
          if (nvis < 128) {                  // V rows behind the query may hold NaN codes, and 0 x NaN is NaN
            ok = mbar_wait_warp(&v_full[st], ph, &s_abort);
            if (!ok) break;
            if (row >= nvis) {
              uint4* vr = reinterpret_cast<uint4*>(ring + st * 2 * ATD8_TILE + ATD8_TILE + row * 128);
#pragma unroll
              for (int i = 0; i < 8; ++i) vr[i] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[ss]);
          ++nb;
          if (++st == ATD8_STAGES) { st = 0; ph ^= 1; }
        }
        if (--left == 0 || bt * 32 + j == n - 1) {         // the (row, group) ends, or this CTA's part of it
          if (need_q) ok = take_q();
          ok = ok && mbar_wait_warp(&us_empty[u & 1], ((u >> 1) & 1) ^ 1, &s_abort);
          if (!ok) break;
          const float ws = warp_reduce16<false>(L, lane);
          if ((lane & 1) == 0) s_l[u & 1][sw][lane >> 1] = ws;
          if (sw == 0 && lane < 16) s_m[u & 1][lane] = mine;
          __syncwarp();
          if (lane == 0) mbar_arrive(&us_full[u & 1]);
          mine = ATD8_LOW;
#pragma unroll
          for (int h = 0; h < 16; ++h) L[h] = 0.f;
          ++u;
          need_q = true;
          left = a.topk;
        }
      }
    }
    if (!left_group) named_bar_any(1, 128, !ok);
  } else {
    // ------------------------------------------------------------ output: thread = dim; the warps run on their own
    const int q4 = warp & 3, dim = q4 * 32 + lane;
    const uint32_t o_addr = tmem + (static_cast<uint32_t>(q4 * 32) << 16) + ATD8_TM_O;
    const int rows = __ldg(a.q_start + a.num_seqs);
    float acc[16];
#pragma unroll
    for (int h = 0; h < 16; ++h) acc[h] = 0.f;
    uint32_t nb = 0;
    int u = 0, left = left0;
    bool ok = true;
    for (int bt = 0; bt < nbatch && ok; ++bt) {
      int4 r;
      uint32_t mask;
      if (!take_batch(bt, r, mask)) break;
      const int cnt = min(32, n - bt * 32);
      for (int j = 0; j < cnt; ++j) {
        if ((mask >> j) & 1) {
          const float vs = __int_as_float(__shfl_sync(0xFFFFFFFFu, r.w, j));
          const uint32_t os = nb % ATD8_RING, par = (nb / ATD8_RING) & 1;
          if (!mbar_wait_warp(&p_full[os], par, &s_abort) || !mbar_wait_warp(&o_full[os], par, &s_abort)) { ok = false; break; }
          tc_fence_after();
          float o[16];
          tmem_ld16(o_addr + os * 16, o);
          float al[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 f = *reinterpret_cast<const float4*>(&s_alpha[os][4 * i]);
            al[4 * i] = f.x; al[4 * i + 1] = f.y; al[4 * i + 2] = f.z; al[4 * i + 3] = f.w;
          }
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_empty[os]);
#pragma unroll
          for (int h = 0; h < 16; ++h) acc[h] = fmaf(o[h], vs, acc[h] * al[h]);
          ++nb;
        }
        const bool last = bt * 32 + j == n - 1;
        if (--left == 0 || last) {
          if (!mbar_wait_warp(&us_full[u & 1], (u >> 1) & 1, &s_abort)) { ok = false; break; }
          const int unit = unit0 + u;
          const int t = unit / a.Hkv, g = unit - t * a.Hkv;
          // whole: the (row, group) lies in this CTA's range; cut ones leave a partial, the CTA's first in part 0
          const bool whole = left == 0 && unit * a.topk >= lo;
          float* part = a.part + (static_cast<long>(blockIdx.x) * 2 + (u ? 1 : 0)) * ATD8_PART;
          if (t < rows) {
#pragma unroll
            for (int h = 0; h < 16; ++h) {
              const float l = (s_l[u & 1][0][h] + s_l[u & 1][1][h]) + (s_l[u & 1][2][h] + s_l[u & 1][3][h]);
              const float m = s_m[u & 1][h];
              if (whole) {
                const long at = static_cast<long>(t) * a.Hq + g * 16 + h;
                a.out[at * 128 + dim] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[h] / l);
                if (a.lse && dim == h) a.lse[at] = l == 0.f ? -INFINITY : (m + (log2f(l) - 8.f)) * 0.69314718055994531f;
              } else {
                part[h * 128 + dim] = acc[h];
                if (dim == h) { part[2048 + h] = m; part[2064 + h] = l; }
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&us_empty[u & 1]);
#pragma unroll
          for (int h = 0; h < 16; ++h) acc[h] = 0.f;
          ++u;
          left = a.topk;
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, ATD8_TMEM);
}

// Joins the parts of a (row, group) that CTA borders cut, in the order of the CTAs (deterministic): with
// W_c = 2^(M_c - max M),  out = sum_c W_c acc_c / sum_c W_c l_c.  CTA = border; it acts if its border is the first inside
// a (row, group).  Thread = (head, 8 dims).
__global__ void __launch_bounds__(256) attn_decode_fp8_merge_kernel(const AttnDecodeFp8Args a, int grid) {
  pdl_wait();                                // the partials of the kernel before, whose end this launch overlaps
  const int c = blockIdx.x + 1;
  const int at = atd8_first(a.n_slots, c, grid), unit = at / a.topk;
  const int first = unit * a.topk, end = first + a.topk;
  const int before = atd8_first(a.n_slots, c - 1, grid);
  if (at == first || before > first) return;
  const int t = unit / a.Hkv, g = unit - t * a.Hkv;
  if (t >= __ldg(a.q_start + a.num_seqs)) return;
  const int h = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * 8;
  const float* p0 = a.part + (static_cast<long>(c - 1) * 2 + (before == first ? 0 : 1)) * ATD8_PART;
  const float* p1 = a.part + static_cast<long>(c) * 2 * ATD8_PART;
  int n = 1;                                 // further parts: CTAs c .. c + n - 1, part 0 of each
  while (c + n < grid && atd8_first(a.n_slots, c + n, grid) < end) ++n;
  auto part = [&](int i) { return i == 0 ? p0 : p1 + static_cast<long>(i - 1) * 2 * ATD8_PART; };
  float mx = ATD8_LOW;
  for (int i = 0; i <= n; ++i) mx = fmaxf(mx, part(i)[2048 + h]);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
#pragma unroll 4
  for (int i = 0; i <= n; ++i) {
    const float* p = part(i);
    const float w = exp2f(p[2048 + h] - mx);
    const float4 x = *reinterpret_cast<const float4*>(p + h * 128 + d0), y = *reinterpret_cast<const float4*>(p + h * 128 + d0 + 4);
    l = fmaf(w, p[2064 + h], l);
    acc[0] = fmaf(w, x.x, acc[0]); acc[1] = fmaf(w, x.y, acc[1]); acc[2] = fmaf(w, x.z, acc[2]); acc[3] = fmaf(w, x.w, acc[3]);
    acc[4] = fmaf(w, y.x, acc[4]); acc[5] = fmaf(w, y.y, acc[5]); acc[6] = fmaf(w, y.z, acc[6]); acc[7] = fmaf(w, y.w, acc[7]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const long o = static_cast<long>(t) * a.Hq + g * 16 + h;
  uint4 r;
  r.x = pack_bf16(acc[0] * inv, acc[1] * inv);
  r.y = pack_bf16(acc[2] * inv, acc[3] * inv);
  r.z = pack_bf16(acc[4] * inv, acc[5] * inv);
  r.w = pack_bf16(acc[6] * inv, acc[7] * inv);
  *reinterpret_cast<uint4*>(a.out + o * 128 + d0) = r;
  if (a.lse && (threadIdx.x & 15) == 0) a.lse[o] = l == 0.f ? -INFINITY : (mx + (log2f(l) - 8.f)) * 0.69314718055994531f;
}

}  // namespace msa
