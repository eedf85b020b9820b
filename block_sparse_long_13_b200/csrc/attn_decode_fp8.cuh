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
// which want Q and P in 8 bits too.  Neither is rounded to 8 bits: each is the sum of a few 8-bit numbers, which are
// columns of one operand and whose products are added in fp32.
//   Q is the sum of two e4m3 numbers, h + l / 16, scaled per head by a power of two so that the largest |q| is in (224, 448].
//      A bf16 number has 8 significant bits; h takes 4 of them, and the rest is a multiple of q's last bit by at most 8 of
//      them either way, which 4 bits hold: exact, down to elements 2^-14 of the head's largest, because the rest is at
//      most 16 and the factor keeps it above e4m3's least step (below them off by 2^-14 of a scaled unit, 2^-21 of the largest
//      element).  Without the factor elements below 2^-10 of it lost bits.
//   P is the sum of three e5m2 numbers (3 significant bits each; the exponents of f16): 2^15 2^(x - m) <= 2^15, m the
//      block's own maximum, as f16 h; then h = p1 + p2 / 8 + p3 / 64, each part the rest of those before it, rounded.  The rests
//      are exact in f16, and the factors 8 and 64 keep them above e5m2's least number for as long as h is normal:
//      off by 2^-11 of itself (f16's 2^-12 included: 2^-10.4) down to probabilities of 2^-29 of the block's largest, by 2^-38
//      of the block's largest below.  A row may put nearly all its weight on one key whose value is near 0 (a sink): its
//      output is then made of the small ones, so what counts is their own size, not the largest one's.  Two e4m3 parts under
//      the row's running maximum, which end at 2^-18 of it, lost a quarter of such an output 12 nats below the sink and all
//      of it from 13.  The sum of probabilities is taken from the unrounded fp32 values.
// Converting the tiles to 16 bits in shared memory instead would read and write 96 KiB of it a block and
// keep a warpgroup busy.
//
// Bound by HBM: 32 KiB a block and group.  148 persistent CTAs, one per SM; each takes an equal run of the
// rows x groups x topk slots, so that every CTA streams the same number of blocks whatever the batch (whole rows per
// CTA would leave 64 x 4 groups two rounds over 148 CTAs: 0.86 busy).  A (row, group) that a border cuts leaves
// partial sums, which attn_decode_fp8_merge_kernel joins.
//
// A block passes through one of ATD8_SLOTS slots, each with its K and V tile, S^T, P^T and O^T; a slot is filled again
// when its O^T has been read, so one full barrier says that everything of the slot is free, and each role waits for
// one barrier a block (a wait for a barrier that is ready takes about 100 clocks, measured, and a block has 1,400).
// Warps: 3 looks up slots (32 at a time: block id, sequence, page, scales) and splits the queries, 0 issues the copies,
// 1 the MMAs of S^T, 2 those of O^T; 4-7 and 12-15 run the softmax on alternate blocks (thread = key; each group keeps
// the running maxima M of its own blocks of the row), 8-11 keep the output of either group's blocks (thread = dim):
// acc = acc 2^(M_old - M) + vs_b 2^(m - M) O_b.  The chain of a block's softmax is longer than the 0.74 us that its 32 KiB
// take at the copy bandwidth (less where rows share blocks): hence two groups.  An MMA as narrow as these takes 47 clocks whatever its N (measured, N <= 64), so the parts are the 16-wide pieces of
// one operand (N = 32 and 48), and the pieces of the result are added when it is read.  Every wait is bounded.
// Measured: 64 rows over 128K keys, 16 blocks, 4 groups: 29.1 to 31.0 us with the merge on two GPUs (134 MB of codes, of which
// rows share some: 116 MB); a block takes 0.66 to 0.74 us a CTA (16 more blocks a row: +20.4 us, 32 more: +36.7), and 10.7 us
// are set-up, first look-ups, first pass through the code and merge; one row over 32K 9.8 to 10.3 us; 32 x 4 verify rows 51.7
// to 53.1 us.  Three parts of P instead of two, and the factor 2^(m - M), cost 0.6 to 1.1 and 2.4 to 2.7 us of that, half of it
// in the softmax and half in the output warps; parts by truncation, or a factor for distant blocks only, changed nothing.
#pragma once
#include "attn_decode.cuh"
#include "e4m3.cuh"
#include "launch_order.cuh"

namespace msa {

constexpr int ATD8_THREADS = 512;
constexpr int ATD8_GRID = 148;         // CTAs at most
constexpr int ATD8_SLOTS = 5;
constexpr int ATD8_TILE = 16384;       // one K or V block: [128 keys][128 dims] codes, 128-byte swizzle
constexpr int ATD8_QT = 4096;          // Q: [high, low][16 heads][128]
constexpr int ATD8_PT = 6144;          // P^T: [16 groups of 8 keys][3 parts][8 keys][16 heads]
constexpr int ATD8_BATCHES = 4;        // slot records in flight, 32 each
constexpr int ATD8_SMEM = ATD8_SLOTS * (2 * ATD8_TILE + ATD8_PT) + 2 * ATD8_QT + 1024;
constexpr uint32_t ATD8_TM_S = 0, ATD8_TM_O = ATD8_SLOTS * 32, ATD8_TMEM = 512;   // 32 and 64 columns each: 16 a part
constexpr int ATD8_PART = 16 * 128 + 32;   // floats of a partial result: sums [16][128], maxima [16], sums of p [16]
constexpr float ATD8_PLOG = 15.f, ATD8_PINV = 0x1p-15f;   // a block's probabilities are held times 2^15
constexpr float ATD8_LOW = -3e38f;     // start of the running maxima (finite: -inf - -inf is NaN)

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
  int num_seqs, Hq, Hkv, topk, max_blocks, num_pages;
  int per, extra;                // slots per CTA; the first `extra` CTAs take one more
  int rows_per_seq;              // total_q / num_seqs, at least 1: where a row's sequence is looked up first
  bool once;                     // tiles are read by one row each
  float scale_log2;
};

// first slot of CTA c
__device__ __forceinline__ int atd8_first(const AttnDecodeFp8Args& a, int c) { return c * a.per + min(c, a.extra); }

// kind::f8f6f4, A e4m3, B e4m3 or e5m2, fp32 accumulate
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn_major, bool b_mn_major, bool b_e5m2 = false) {
  return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void umma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// descriptor of P^T, an unswizzled MN-major 8-bit operand of three 16-wide parts: 8 x 16 byte core matrices, the parts
// 128 bytes and the groups of 8 keys 384 bytes apart
__device__ __forceinline__ uint64_t sdesc_pt(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(384 >> 4) << 16) |
         (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

// mbar_wait that polls for a while before it goes to the clock, out of line: the timer and the limit's global load
// would make every short wait late, and the copies of that code fill the instruction cache.
__device__ __noinline__ bool mbar_wait_long(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_wait(bar, parity, abort);
}
__device__ __forceinline__ bool mbar_wait_soon(uint64_t* bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait_long(bar, parity, abort);
}
__device__ __forceinline__ bool mbar_wait_soon_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const bool ok = mbar_wait_soon(bar, parity, abort);
  return !__any_sync(0xFFFFFFFFu, !ok);
}

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// two values (<= 448 in size) as e4m3 pairs, a = hi + lo / 16
__device__ __forceinline__ void e4m3x2_split(float a, float b, uint32_t& hi, uint32_t& lo) {
  uint32_t h2, back, d;
  uint16_t u, v;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h2) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(u) : "r"(h2));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h2), "r"(back));
  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(d) : "r"(0x4C004C00u));   // 16
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(v) : "r"(d));
  hi = u;
  lo = v;
}

// Two values (0 .. 2^15) as three pairs of e5m2 numbers, a = a1 + a2 / 8 + a3 / 64: an e5m2 number is the upper byte of an f16
// one, so the first two pairs are left there (their lower bytes are 0), and half a step added to the bits rounds to it.  A NaN
// (0x7FFF) loses itself in that sum but not in the rests, and arrives in the third part.
__device__ __forceinline__ void e5m2x2_split(float a, float b, uint32_t& p1, uint32_t& p2, uint32_t& p3) {
  uint32_t h, d;
  uint16_t u;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(b), "f"(a));
  p1 = (h + 0x00800080u) & 0xFF00FF00u;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h), "r"(p1));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h) : "r"(d), "r"(0x48004800u));   // 8
  p2 = (h + 0x00800080u) & 0xFF00FF00u;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h), "r"(p2));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h) : "r"(d), "r"(0x48004800u));
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(u) : "r"(h));
  p3 = u;
}

// A head's queries come to (224, 448] times 2^k, 448 = 1.75 * 2^8, by the largest of them (|q| as bf16 bits: NaN above
// infinity above the rest).
__device__ __forceinline__ uint32_t abs_max_bf16(const uint4& x) {
  const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
  return max(m & 0xFFFFu, m >> 16);
}
__device__ __forceinline__ int query_exponent(uint32_t m) {
  return min(120, 135 - static_cast<int>(m >> 7) - ((m & 0x7Fu) > 0x60u ? 1 : 0));
}
// what the scores of such a head are multiplied by; an infinite or NaN query makes its head NaN
__device__ __forceinline__ float query_factor(uint32_t m, float scale_log2) {
  return m >= 0x7F80u ? __uint_as_float(0x7FC00000u)
                      : scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - query_exponent(m)) << 23);
}
// 16 dims (two 16-byte loads) from dim d on of head h into the parts of the Q tile
__device__ __forceinline__ void split_queries(uint8_t* qt, int h, int d, const uint4& x, const uint4& y, float mult) {
  const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  uint32_t hi[4], lw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h0, l0, h1, l1;
    e4m3x2_split(bf16lo(w[2 * i]) * mult, bf16hi(w[2 * i]) * mult, h0, l0);
    e4m3x2_split(bf16lo(w[2 * i + 1]) * mult, bf16hi(w[2 * i + 1]) * mult, h1, l1);
    hi[i] = h0 | (h1 << 16);
    lw[i] = l0 | (l1 << 16);
  }
  const uint32_t at = sw128_offset(h, d);
  *reinterpret_cast<uint4*>(qt + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  *reinterpret_cast<uint4*>(qt + 2048 + at) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
}

// The sequence of row t: exact at the first look when all sequences have as many rows, a search otherwise.
__device__ __forceinline__ int find_seq_even(const int32_t* q_start, int num_seqs, int rows_per_seq, int t) {
  const int s = min(num_seqs - 1, t / rows_per_seq);
  if (__ldg(q_start + s) <= t && t < __ldg(q_start + s + 1)) return s;
  return find_seq(q_start, num_seqs, t);
}

__global__ void __launch_bounds__(ATD8_THREADS, 1)
attn_decode_fp8_kernel(const __grid_constant__ CUtensorMap tmap_k,    // k codes as [P*Hkv*128][128]
                       const __grid_constant__ CUtensorMap tmap_v, const AttnDecodeFp8Args a) {
  extern __shared__ __align__(1024) uint8_t dsmem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
  uint8_t* tiles = smem;                                  // slots of [K 16 KiB][V 16 KiB]
  uint8_t* q_s = tiles + ATD8_SLOTS * 2 * ATD8_TILE;      // 2 x [high, low][16 heads][128] (128-byte swizzle)
  uint8_t* p_s = q_s + 2 * ATD8_QT;                       // slots of P^T

  // Of a slot: kv_full its tiles are there; s_full S^T is in TMEM; p_full P^T and the factors are in shared memory;
  // o_full O^T is in TMEM; o_empty O^T and the factors are read.
  __shared__ uint64_t kv_full[ATD8_SLOTS], s_full[ATD8_SLOTS], p_full[ATD8_SLOTS], o_full[ATD8_SLOTS],
      o_empty[ATD8_SLOTS], rec_full[ATD8_BATCHES], rec_empty[ATD8_BATCHES], q_full[2], q_empty[2], us_full[2],
      us_empty[2], drain_bar[2];
  __shared__ __align__(16) int4 s_rec[ATD8_BATCHES * 32]; // slot: TMA row or -1, visible keys, K scale, V scale
  __shared__ uint32_t s_mask[ATD8_BATCHES];               // slots of the batch that hold a block
  __shared__ __align__(16) float s_fq[2][16];             // softmax scale x log2 e / the query's power of two
  __shared__ __align__(16) float s_red[2][2][4][16];      // per softmax group: the warps' maxima of a block, by parity
  __shared__ __align__(16) float s_run[8][3][16];         // per softmax warp: a block's maxima m, 2^(M_old - M), 2^(m - M - 15)
  __shared__ __align__(16) float s_fac[ATD8_SLOTS][2][16];   // 2^(M_old - M) and 2^(m - M) of a block
  __shared__ __align__(16) float s_m[2][2][16], s_l[2][8][16];   // of a finished (row, group): maxima, sums of p per warp
  __shared__ __align__(16) float s_fin[4][2][16];         // per output warp: what the two groups' sums are weighted by
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lo = atd8_first(a, blockIdx.x);
  const int n = atd8_first(a, blockIdx.x + 1) - lo;       // > 0: no more CTAs than slots
  const int nbatch = (n + 31) >> 5;
  const int unit0 = lo / a.topk;
  const int left0 = a.topk - (lo - unit0 * a.topk);       // slots of the first (row, group) in this range
  if (warp == 0) {
    pdl_launch_dependents();
    if (lane == 0) s_abort = 0;
    if (lane < ATD8_SLOTS) {
      mbar_init(&kv_full[lane], 1);
      mbar_init(&s_full[lane], 1);
      mbar_init(&p_full[lane], 4);
      mbar_init(&o_full[lane], 1);
      mbar_init(&o_empty[lane], 4);
    }
    if (lane < ATD8_BATCHES) {
      mbar_init(&rec_full[lane], 1);
      mbar_init(&rec_empty[lane], 15);                    // producer, two issuers, 8 softmax and 4 output warps
    }
    if (lane < 2) {
      mbar_init(&q_full[lane], 1);
      mbar_init(&q_empty[lane], 9);                       // issuer, 8 softmax warps
      mbar_init(&us_full[lane], 8);
      mbar_init(&us_empty[lane], 4);
      mbar_init(&drain_bar[lane], 1);
    }
    fence_mbar_init();
    __syncwarp();
    if (lane == 0) {                         // the first records and queries are written before the block's barrier below
      mbar_arrive(&rec_full[0]);
      mbar_arrive(&q_full[0]);
    }
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, ATD8_TMEM);
    tmem_relinquish();
  }
  // The record of slot lane of batch bt: block id and sequence, then position and page, then the scales, a round trip
  // each.
  auto look_up = [&](int bt) -> int4 {
    int4 rec = make_int4(-1, 0, 0, 0);
    const int i = lo + bt * 32 + lane;
    if (bt * 32 + lane < n) {
      const int b = __ldg(a.block_idx + i);
      const int unit = i / a.topk, t = unit / a.Hkv, g = unit - t * a.Hkv;
      const int s = find_seq_even(a.q_start, a.num_seqs, a.rows_per_seq, t);
      const int end = __ldg(a.q_start + s + 1), ctx = __ldg(a.ctx_len + s);
      const bool listed = b >= 0 && b < a.max_blocks;
      const int page = listed ? __ldg(a.page_table + static_cast<long>(s) * a.max_blocks + b) : -1;
      if (b >= 0 && t < end) {                            // rows behind the last sequence hold nothing
        const int p = ctx - end + t;
        if (page >= 0 && page < a.num_pages && b * 128 <= p) {
          const int tile = page * a.Hkv + g;
          rec = make_int4(tile * 128, min(128, p - b * 128 + 1), __float_as_int(__ldg(a.k_scale + tile)),
                          __float_as_int(__ldg(a.v_scale + tile)));
        } else {
          flag_error(MSA_DEV_BOUNDS);
        }
      }
    }
    return rec;
  };
  auto q_row = [&](int unit, int h) {
    const int t = unit / a.Hkv, g = unit - t * a.Hkv;
    return reinterpret_cast<const uint4*>(a.q + (static_cast<long>(t) * a.Hq + g * 16 + h) * 128);
  };
  auto put_batch = [&](int rb, const int4& rec) {
    s_rec[rb * 32 + lane] = rec;
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, rec.x >= 0);
    if (lane == 0) s_mask[rb] = mask;
  };
  // While the barriers are set up: the first records (warp 3) and the first queries (warps 8-11, 8 threads a head).
  if (warp == 3) {
    put_batch(0, look_up(0));
  } else if (warp >= 8 && warp < 12) {
    const int h = (tid - 256) >> 3, d8 = tid & 7;
    const uint4 x = __ldg(q_row(unit0, h) + 2 * d8), y = __ldg(q_row(unit0, h) + 2 * d8 + 1);
    uint32_t m = max(abs_max_bf16(x), abs_max_bf16(y));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    split_queries(q_s, h, d8 * 16, x, y, __uint_as_float(static_cast<uint32_t>(127 + query_exponent(m)) << 23));
    if (d8 == 0) s_fq[0][h] = query_factor(m, a.scale_log2);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // The records of batch bt: lane's slot, and which of the batch's slots hold a block.  Warp-uniform result.
  auto take_batch = [&](int bt, int4& r, uint32_t& mask) -> bool {
    const int rb = bt & (ATD8_BATCHES - 1);
    if (!mbar_wait_soon_warp(&rec_full[rb], (bt / ATD8_BATCHES) & 1, &s_abort)) return false;
    r = s_rec[rb * 32 + lane];
    mask = s_mask[rb];
    __syncwarp();
    if (lane == 0) mbar_arrive(&rec_empty[rb]);
    return true;
  };

  if (warp == 3) {
    // ------------------------------------------------------------ slot records, and the queries of the rows they begin
    // A batch's records go out before the queries of its (row, group)s are waited for: what those waits need (the
    // (row, group) two before, its blocks and its queries) is out by then.
    const int nu = (lo + n - 1) / a.topk - unit0 + 1;
    const int h = lane >> 1, half = lane & 1;             // queries: half a head a lane
    int u = 1;
    uint4 x[8];
    auto load_q = [&]() {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __ldg(q_row(unit0 + u, h) + half * 8 + i);
    };
    if (nu > 1) load_q();
    for (int bt = 0; bt < nbatch; ++bt) {
      if (bt > 0) {
        const int4 rec = look_up(bt);
        const int rb = bt & (ATD8_BATCHES - 1);
        if (!mbar_wait_soon_warp(&rec_empty[rb], ((bt / ATD8_BATCHES) & 1) ^ 1, &s_abort)) break;
        put_batch(rb, rec);
        __syncwarp();
        if (lane == 0) mbar_arrive(&rec_full[rb]);
      }
      const int begun = min(nu, (lo + min(n, bt * 32 + 32) - 1) / a.topk - unit0 + 1);   // (row, group)s begun so far
      for (; u < begun; ++u) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, abs_max_bf16(x[i]));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        const float mult = __uint_as_float(static_cast<uint32_t>(127 + query_exponent(m)) << 23);
        const int qb = u & 1;
        if (!mbar_wait_soon_warp(&q_empty[qb], ((u >> 1) & 1) ^ 1, &s_abort)) { bt = nbatch; break; }
        if (half == 0) s_fq[qb][h] = query_factor(m, a.scale_log2);
#pragma unroll
        for (int i = 0; i < 4; ++i) split_queries(q_s + qb * ATD8_QT, h, half * 64 + i * 16, x[2 * i], x[2 * i + 1], mult);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[qb]);
        if (u + 1 < nu) {
          ++u;
          load_q();
          --u;
        }
      }
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
        if (!mbar_wait_soon_warp(&o_empty[st], ph, &s_abort)) { ok = false; break; }
        if (lane == 0) {
          uint8_t* dst = tiles + st * 2 * ATD8_TILE;
          mbar_arrive_expect_tx(&kv_full[st], 2 * ATD8_TILE);
          if (a.once) {
            tma_load_2d_hint(dst, &tmap_k, &kv_full[st], 0, row, pol);
            tma_load_2d_hint(dst + ATD8_TILE, &tmap_v, &kv_full[st], 0, row, pol);
          } else {
            tma_load_2d(dst, &tmap_k, &kv_full[st], 0, row);
            tma_load_2d(dst + ATD8_TILE, &tmap_v, &kv_full[st], 0, row);
          }
        }
        ++used;
        if (++st == ATD8_SLOTS) { st = 0; ph ^= 1; }
      }
    }
    if (lane == 0 && s_abort)                // let every issued copy land before the CTA exits
      for (int i = 0; i < ATD8_SLOTS && i < used; ++i) mbar_wait_drain(&kv_full[i], ((used - 1 - i) / ATD8_SLOTS) & 1);
  } else if (warp == 1) {
    // ------------------------------------------------------------ S^T = K_b Q^T; lane 0 issues
    const uint32_t id_s = idesc_e4m3(128, 32, false, false);   // A = K_b (K-major), B = Q (K-major)
    const uint64_t k_d = sdesc_sw128(smem_u32(tiles), 16, 1024);
    const uint64_t q_d = sdesc_sw128(smem_u32(q_s), 16, 1024);
    int st = 0, ph = 0, left = left0, u = 0;
    bool ok = true, begin = true;
    for (int bt = 0; bt < nbatch && ok; ++bt) {
      int4 r;
      uint32_t mask;
      if (!take_batch(bt, r, mask)) break;
      const int cnt = min(32, n - bt * 32);
      for (int j = 0; j < cnt; ++j) {
        if (begin && !mbar_wait_soon(&q_full[u & 1], (u >> 1) & 1, &s_abort)) { ok = false; break; }
        begin = false;
        if ((mask >> j) & 1) {
          if (!mbar_wait_soon(&kv_full[st], ph, &s_abort)) { ok = false; break; }
          tc_fence_after();
          if (lane == 0) {
            const uint64_t kd = k_d + ((st * 2 * ATD8_TILE) >> 4), qd = q_d + (((u & 1) * ATD8_QT) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)   // 32 dims per step, within a 128-byte row
              umma_f8_ss(tmem + ATD8_TM_S + st * 32, kd + kk * 2, qd + kk * 2, id_s, kk > 0 ? 1u : 0u);
            umma_commit(&s_full[st]);
          }
          if (++st == ATD8_SLOTS) { st = 0; ph ^= 1; }
        }
        if (--left == 0 || bt * 32 + j == n - 1) {
          if (lane == 0) umma_commit(&q_empty[u & 1]);
          ++u;
          begin = true;
          left = a.topk;
        }
      }
      ok = !__any_sync(0xFFFFFFFFu, !ok);
    }
    if (lane == 0 && s_abort) {
      umma_commit(&drain_bar[0]);
      mbar_wait_drain(&drain_bar[0], 0);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ O_b^T = V_b^T P^T; lane 0 issues
    const uint32_t id_pv = idesc_e4m3(128, 48, true, true, true);   // A = V_b^T, B = P^T in e5m2 (both MN-major)
    const uint64_t v_d = sdesc_sw128(smem_u32(tiles) + ATD8_TILE, ATD8_TILE, 1024);
    const uint64_t p_d = sdesc_pt(smem_u32(p_s));
    int st = 0, ph = 0;
    bool ok = true;
    for (int bt = 0; bt < nbatch && ok; ++bt) {
      int4 r;
      uint32_t mask;
      if (!take_batch(bt, r, mask)) break;
      for (; mask; mask &= mask - 1) {
        if (!mbar_wait_soon(&p_full[st], ph, &s_abort)) { ok = false; break; }
        tc_fence_after();
        if (lane == 0) {
          const uint64_t vd = v_d + ((st * 2 * ATD8_TILE) >> 4), pd = p_d + ((st * ATD8_PT) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)     // 32 keys per step: 4 KiB of V rows, 1.5 KiB of P rows
            umma_f8_ss(tmem + ATD8_TM_O + st * 64, vd + kk * 256, pd + kk * 96, id_pv, kk > 0 ? 1u : 0u);
          umma_commit(&o_full[st]);
        }
        if (++st == ATD8_SLOTS) { st = 0; ph ^= 1; }
      }
      ok = !__any_sync(0xFFFFFFFFu, !ok);
    }
    if (lane == 0 && s_abort) {
      umma_commit(&drain_bar[1]);
      mbar_wait_drain(&drain_bar[1], 0);
    }
  } else if (warp < 8 || warp > 11) {
    // ------------------------------------------------------------ softmax: thread = key
    // Group 0 (warps 4-7) takes the CTA's even blocks, group 1 (warps 12-15) the odd ones.  A group's four warps meet
    // at one barrier a block (the exchange of their maxima), which also carries a failed wait to all of them: after a
    // failed wait a warp goes to that barrier and leaves, and so do the others there or at the last barrier, behind
    // the last slot.
    const int grp = warp > 11 ? 1 : 0, sw = warp & 3, row = sw * 32 + lane;   // sw: the TMEM quarter of the warp
    const int w8 = grp * 4 + sw, h16 = lane & 15;
    const uint32_t s_addr = tmem + (static_cast<uint32_t>(sw * 32) << 16) + ATD8_TM_S;
    // Lane h (and h + 16) keeps the running maximum of head h; the sums are per thread, i.e. per key.
    float mine = ATD8_LOW, L[16], fq[16];
#pragma unroll
    for (int h = 0; h < 16; ++h) L[h] = fq[h] = 0.f;
    int st = 0, ph = 0, left = left0, u = 0;
    uint32_t nb = 0;
    bool ok = true, met = false, begin = true;
    for (int bt = 0; bt < nbatch && ok && !met; ++bt) {
      int4 r;
      uint32_t mask;
      if (!take_batch(bt, r, mask)) { ok = false; break; }
      const int cnt = min(32, n - bt * 32);
#pragma unroll 1
      for (int j = 0; j < cnt; ++j) {
        if (begin) {                         // a (row, group) begins: its queries' scales
          begin = false;
          if (!mbar_wait_soon_warp(&q_full[u & 1], (u >> 1) & 1, &s_abort)) { ok = false; break; }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 f = *reinterpret_cast<const float4*>(&s_fq[u & 1][4 * i]);
            fq[4 * i] = f.x; fq[4 * i + 1] = f.y; fq[4 * i + 2] = f.z; fq[4 * i + 3] = f.w;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_empty[u & 1]);
        }
        const bool block = (mask >> j) & 1;
        if (block && static_cast<int>(nb & 1) == grp) {
          const int nvis = __shfl_sync(0xFFFFFFFFu, r.y, j);
          const float ks = __int_as_float(__shfl_sync(0xFFFFFFFFu, r.z, j));
          ok = mbar_wait_soon(&s_full[st], ph, &s_abort);   // a failure is shared at the barrier below
          __syncwarp();
          tc_fence_after();
          float v[32], x[16];
          tmem_ld32(s_addr + st * 32, v);
          tmem_ld_wait();
          tc_fence_before();
#pragma unroll
          for (int h = 0; h < 16; ++h) x[h] = fmaf(v[16 + h], 0.0625f, v[h]) * (fq[h] * ks);
          if (row >= nvis) {                 // keys behind the query's position do not count
#pragma unroll
            for (int h = 0; h < 16; ++h) x[h] = -INFINITY;
          }
          __syncwarp();
          float (&red)[4][16] = s_red[grp][(nb >> 1) & 1];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 wm = make_float4(warp_max(x[4 * i]), warp_max(x[4 * i + 1]), warp_max(x[4 * i + 2]), warp_max(x[4 * i + 3]));
            if (lane == 0) *reinterpret_cast<float4*>(&red[sw][4 * i]) = wm;
          }
          if (named_bar_any(1 + grp, 128, !ok)) { met = true; break; }
          // every warp joins the four maxima for itself, a head per lane, and hands them to its lanes
          const float bm = fmaxf(fmaxf(fmaxf(red[0][h16], red[1][h16]), fmaxf(red[2][h16], red[3][h16])), ATD8_LOW);
          const float old = mine;
          mine = fmaxf(old, bm);
          const float fac = exp2f(old - mine), rel = exp2f(bm - mine);
          if (lane < 16) {
            s_run[w8][0][lane] = bm;
            s_run[w8][1][lane] = fac;
            s_run[w8][2][lane] = rel * ATD8_PINV;
            if (sw == 0) {
              s_fac[st][0][lane] = fac;
              s_fac[st][1][lane] = rel;
            }
          }
          if (__any_sync(0xFFFFFFFFu, mine > old)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 f = *reinterpret_cast<const float4*>(&s_run[w8][1][4 * i]);
              L[4 * i] *= f.x; L[4 * i + 1] *= f.y; L[4 * i + 2] *= f.z; L[4 * i + 3] *= f.w;
            }
          }
          __syncwarp();
          uint32_t p1[4], p2[4], p3[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 m = *reinterpret_cast<const float4*>(&s_run[w8][0][4 * i]);
            const float4 f = *reinterpret_cast<const float4*>(&s_run[w8][2][4 * i]);
            const float mm[4] = {m.x, m.y, m.z, m.w}, ff[4] = {f.x, f.y, f.z, f.w};
            float p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              p[k] = exp2f((x[4 * i + k] - mm[k]) + ATD8_PLOG);        // 2^15 2^(x - m); 2^-inf = 0
              L[4 * i + k] = fmaf(p[k], ff[k], L[4 * i + k]);
            }
            uint32_t a1, a2, a3, b1, b2, b3;
            e5m2x2_split(p[0], p[1], a1, a2, a3);
            e5m2x2_split(p[2], p[3], b1, b2, b3);
            p1[i] = __byte_perm(a1, b1, 0x7531);
            p2[i] = __byte_perm(a2, b2, 0x7531);
            p3[i] = a3 | (b3 << 16);
          }
          uint8_t* pt = p_s + st * ATD8_PT + (row >> 3) * 384 + (row & 7) * 16;
          *reinterpret_cast<uint4*>(pt) = make_uint4(p1[0], p1[1], p1[2], p1[3]);
          *reinterpret_cast<uint4*>(pt + 128) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
          *reinterpret_cast<uint4*>(pt + 256) = make_uint4(p3[0], p3[1], p3[2], p3[3]);
          if (nvis < 128) {                  // V rows behind the query may hold NaN codes, and 0 x NaN is NaN
            if (!mbar_wait_soon_warp(&kv_full[st], ph, &s_abort)) { ok = false; break; }
            if (row >= nvis) {
              uint4* vr = reinterpret_cast<uint4*>(tiles + st * 2 * ATD8_TILE + ATD8_TILE + row * 128);
#pragma unroll
              for (int i = 0; i < 8; ++i) vr[i] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[st]);
        }
        if (block) {
          ++nb;
          if (++st == ATD8_SLOTS) { st = 0; ph ^= 1; }
        }
        if (--left == 0 || bt * 32 + j == n - 1) {         // the (row, group) ends, or this CTA's part of it
          if (!mbar_wait_soon_warp(&us_empty[u & 1], ((u >> 1) & 1) ^ 1, &s_abort)) { ok = false; break; }
          const float ws = warp_reduce16<false>(L, lane);
          if ((lane & 1) == 0) s_l[u & 1][w8][lane >> 1] = ws;
          if (sw == 0 && lane < 16) s_m[u & 1][grp][lane] = mine;
          __syncwarp();
          if (lane == 0) mbar_arrive(&us_full[u & 1]);
          mine = ATD8_LOW;
#pragma unroll
          for (int h = 0; h < 16; ++h) L[h] = 0.f;
          ++u;
          begin = true;
          left = a.topk;
        }
      }
    }
    if (!met) named_bar_any(1 + grp, 128, !ok);
  } else {
    // ------------------------------------------------------------ output: thread = dim; the warps run on their own
    const int q4 = warp & 3, dim = q4 * 32 + lane;
    const uint32_t o_addr = tmem + (static_cast<uint32_t>(q4 * 32) << 16) + ATD8_TM_O;
    const int rows = __ldg(a.q_start + a.num_seqs);
    float acc0[16], acc1[16];                // of the even and of the odd blocks
#pragma unroll
    for (int h = 0; h < 16; ++h) acc0[h] = acc1[h] = 0.f;
    int st = 0, ph = 0, left = left0, u = 0;
    uint32_t nb = 0;
    bool ok = true;
    for (int bt = 0; bt < nbatch && ok; ++bt) {
      int4 r;
      uint32_t mask;
      if (!take_batch(bt, r, mask)) break;
      const int cnt = min(32, n - bt * 32);
#pragma unroll 1
      for (int j = 0; j < cnt; ++j) {
        if ((mask >> j) & 1) {
          const float vs = __int_as_float(__shfl_sync(0xFFFFFFFFu, r.w, j));
          if (!mbar_wait_soon_warp(&o_full[st], ph, &s_abort)) { ok = false; break; }
          tc_fence_after();
          float o[16], o2[16], o3[16], al[16], f[16];
          tmem_ld16(o_addr + st * 64, o);
          tmem_ld16(o_addr + st * 64 + 16, o2);
          tmem_ld16(o_addr + st * 64 + 32, o3);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(&s_fac[st][0][4 * i]);
            const float4 y = *reinterpret_cast<const float4*>(&s_fac[st][1][4 * i]);
            al[4 * i] = x.x; al[4 * i + 1] = x.y; al[4 * i + 2] = x.z; al[4 * i + 3] = x.w;
            f[4 * i] = y.x * vs; f[4 * i + 1] = y.y * vs; f[4 * i + 2] = y.z * vs; f[4 * i + 3] = y.w * vs;
          }
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_empty[st]);
#pragma unroll
          for (int h = 0; h < 16; ++h) o[h] = fmaf(fmaf(o3[h], 0.125f, o2[h]), 0.125f * ATD8_PINV, o[h] * ATD8_PINV);
          if (nb & 1) {
#pragma unroll
            for (int h = 0; h < 16; ++h) acc1[h] = fmaf(o[h], f[h], acc1[h] * al[h]);
          } else {
#pragma unroll
            for (int h = 0; h < 16; ++h) acc0[h] = fmaf(o[h], f[h], acc0[h] * al[h]);
          }
          ++nb;
          if (++st == ATD8_SLOTS) { st = 0; ph ^= 1; }
        }
        if (--left == 0 || bt * 32 + j == n - 1) {
          if (!mbar_wait_soon_warp(&us_full[u & 1], (u >> 1) & 1, &s_abort)) { ok = false; break; }
          const int unit = unit0 + u;
          const int t = unit / a.Hkv, g = unit - t * a.Hkv;
          // whole: the (row, group) lies in this CTA's range; cut ones leave a partial, the CTA's first in part 0
          const bool whole = left == 0 && unit * a.topk >= lo, valid = t < rows;
          float* part = a.part + (static_cast<long>(blockIdx.x) * 2 + (u ? 1 : 0)) * ATD8_PART;
          const long head0 = static_cast<long>(t) * a.Hq + g * 16;
          if (lane < 16) {                   // a head per lane: the groups' weights, over the sum where it is complete
            const float(&sl)[8][16] = s_l[u & 1];
            const float m0 = s_m[u & 1][0][lane], m1 = s_m[u & 1][1][lane], m = fmaxf(m0, m1);
            const float w0 = exp2f(m0 - m), w1 = exp2f(m1 - m);
            const float l = w0 * ((sl[0][lane] + sl[1][lane]) + (sl[2][lane] + sl[3][lane])) +
                            w1 * ((sl[4][lane] + sl[5][lane]) + (sl[6][lane] + sl[7][lane]));
            const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
            s_fin[q4][0][lane] = w0 * inv;
            s_fin[q4][1][lane] = w1 * inv;
            if (q4 == 0 && valid) {
              if (!whole) {
                part[2048 + lane] = m;
                part[2064 + lane] = l;
              } else if (a.lse) {
                a.lse[head0 + lane] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&us_empty[u & 1]);
          if (valid) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 f0 = *reinterpret_cast<const float4*>(&s_fin[q4][0][4 * i]);
              const float4 f1 = *reinterpret_cast<const float4*>(&s_fin[q4][1][4 * i]);
              const float y[4] = {acc0[4 * i] * f0.x + acc1[4 * i] * f1.x, acc0[4 * i + 1] * f0.y + acc1[4 * i + 1] * f1.y,
                                  acc0[4 * i + 2] * f0.z + acc1[4 * i + 2] * f1.z, acc0[4 * i + 3] * f0.w + acc1[4 * i + 3] * f1.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (whole) a.out[(head0 + 4 * i + k) * 128 + dim] = __float2bfloat16_rn(y[k]);
                else part[(4 * i + k) * 128 + dim] = y[k];
              }
            }
          }
          __syncwarp();                      // s_fin is written again at the next (row, group)
#pragma unroll
          for (int h = 0; h < 16; ++h) acc0[h] = acc1[h] = 0.f;
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
// a (row, group).  A CTA takes four heads (a whole (row, group) of 16 parts is 128 KiB, more than one SM reads in
// 2 us), a warp a head, a lane 4 dims; four parts are in flight (sixteen, in registers, took as long).
__global__ void __launch_bounds__(128) attn_decode_fp8_merge_kernel(const AttnDecodeFp8Args a, int grid) {
  const int c = (blockIdx.x >> 2) + 1;
  const int at = atd8_first(a, c), unit = at / a.topk;
  const int first = unit * a.topk, end = first + a.topk;
  const int before = atd8_first(a, c - 1);
  const int t = unit / a.Hkv, g = unit - t * a.Hkv;
  const bool acts = at != first && before <= first && t < __ldg(a.q_start + a.num_seqs);
  // parts: of CTA c - 1, then part 0 of the CTAs c .. that begin inside the (row, group)
  int n = 2;
  if (acts)
    while (c + n - 1 < grid && atd8_first(a, c + n - 1) < end) ++n;
  const int h = (blockIdx.x & 3) * 4 + (threadIdx.x >> 5), d0 = (threadIdx.x & 31) * 4;
  const float* p0 = a.part + static_cast<long>(c - 1) * 2 * ATD8_PART;
  pdl_wait();                                // the partials of the kernel before, whose end this launch overlaps
  if (!acts) return;
  float M = ATD8_LOW, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    // CTA c - 1 may have begun before the (row, group): its part 1
    const float* p = p0 + (i == 0 && before != first ? 1 : 2 * i) * ATD8_PART;
    const float m = p[2048 + h], lw = p[2064 + h];
    const float4 x = *reinterpret_cast<const float4*>(p + h * 128 + d0);
    const float mx = fmaxf(M, m), al = exp2f(M - mx), w = exp2f(m - mx);
    M = mx;
    l = fmaf(w, lw, l * al);
    acc.x = fmaf(w, x.x, acc.x * al); acc.y = fmaf(w, x.y, acc.y * al);
    acc.z = fmaf(w, x.z, acc.z * al); acc.w = fmaf(w, x.w, acc.w * al);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const long o = static_cast<long>(t) * a.Hq + g * 16 + h;
  *reinterpret_cast<uint2*>(a.out + o * 128 + d0) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (a.lse && d0 == 0) a.lse[o] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
}

}  // namespace msa
