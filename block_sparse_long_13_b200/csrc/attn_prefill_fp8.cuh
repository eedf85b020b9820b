// msa_attn_prefill_fp8: block-major sparse GQA attention over a paged cache of e4m3 codes with one fp32 scale for each
// (page, KV head).
//
// The block-major form of attn_prefill.cuh (a tile stacks the 16 heads of up to 8 tokens that selected the block;
// S = Q K^T and O = P V on tcgen05; per-slot partials; log-sum-exp merge), over codes:
//   x_j = (scale log2 e) ks_b (q . ck_j),   O_b = vs_b sum_j 2^(x_j - m) cv_j / l,   lse_b = (m + log2 l) ln 2.
// The codes are widened once per (run of tiles, block) by four converter warps, K to bf16 (an MMA's operands have one
// type, and the queries are bf16) and V to f16, times 2^-15 (P is then f16 too, three bits more than bf16); both hold every
// e4m3 value.  The scales stay fp32 factors of the softmax and of the output: nothing is rounded that the bf16 form does not
// round.  P is 2^14 times the probability relative to the block's largest, for which V's 2^-15 makes room: f16 holds it to
// 2^-12 of itself down to 2^-28 of the largest.  A key of large weight and a value near 0 (a sink) leaves the output to the
// small ones, and with P at most 1/2 those 15 nats below it were off by 2 % and lost from 17.
// Feeding the tensor cores with the codes, as the decode form does, would take P in two 8-bit parts, 256 more
// instructions for each row of 128 keys in the softmax warps that set this kernel's pace; a block's widening is 20 to 45
// instructions per 16 codes, once for all tokens that selected it, in warps of their own.
//
// Bound by the chain of a tile's steps: two softmax groups take tiles in turn, a pair of tiles 6,000 clocks (scores out of
// TMEM 430, exponentials 1,530, P V 1,100 to 1,800, output 1,400, waits), of which the tensor cores are held for 3,400 and
// DRAM for a third.  What shortened it: records through shared memory instead of global loads whose use the registers'
// allocation moved behind the loop (2.65 -> 2.58 ms), partials without the division and the part's statistics behind the
// stores (2.42), S and P V issued by two threads (mixed chunks 239 -> 230 us), K and V in two buffers each, for which the
// partials go straight from the registers to memory instead of by way of shared memory (230 -> 221 and 2.42 ms alike; that
// alone, with one buffer: 235 and 2.58).  V's factor and the rare forms (NaN codes, huge scores) cost 221 -> 228.  P handed over
// in halves changed nothing.  The last 16,384 rows of 128K take 2.4
// ms: schedule 0.04, tiles 1.64 (670 TFLOP/s of S and P V), merge 0.68 at 6.4 TB/s.
#pragma once
#include "attn_prefill.cuh"
#include "e4m3.cuh"
#include "launch_order.cuh"

namespace msa {

// Warpgroup 0: producer and issuer warps; 1: converters; 2, 3: softmax.  Register split (setmaxnreg) of the launch's
// 128 a thread: 128 * (56 + 88 + 184 + 184) = 65536.
constexpr int ATP8_THREADS = 512;
constexpr int ATP8_QBUF = 3;     // gathered query tiles in flight
constexpr int ATP8_SMEM = ATP8_QBUF * ATTP_QBYTES + 4 * ATTP_KVBYTES + 1024;
constexpr int ATP8_RECS = 8;     // ring of records
constexpr int ATP8_RUN = 64;     // tiles of a CTA and round
constexpr int ATP8_REGS_CTRL = 56, ATP8_REGS_CONV = 88, ATP8_REGS_SOFTMAX = 184;
static_assert(ATP8_REGS_CTRL + ATP8_REGS_CONV + 2 * ATP8_REGS_SOFTMAX <= 4 * 128, "register split exceeds the launch");

// ------------------------------------------------------------------ codes to bf16
// whether one of 16 codes is NaN (0x7F or 0xFF)
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ bool has_nan(const uint4& x) {
  return (nan_bytes(x.x) | nan_bytes(x.y) | nan_bytes(x.z) | nan_bytes(x.w)) != 0u;
}
__device__ __forceinline__ uint4 without_nan(uint4 x) {   // NaN codes become 0
  auto clear = [](uint32_t w) { const uint32_t b = nan_bytes(w) >> 7; return w & ~(b * 0xFFu); };
  return make_uint4(clear(x.x), clear(x.y), clear(x.z), clear(x.w));
}
// whether there is one among the codes of a warp
__device__ __forceinline__ bool warp_has_nan(const uint4 (&x)[8]) {
  uint32_t any = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) any |= nan_bytes(x[k].x) | nan_bytes(x[k].y) | nan_bytes(x[k].z) | nan_bytes(x[k].w);
  return __any_sync(0xFFFFFFFFu, any != 0u);
}
// Two codes (bytes 1 and 3 of t) as bf16: exponent and mantissa move to bits 10..4, where they stand for the code's
// value times 2^-120 (bias 127 instead of 7; subnormals too), and a product with 2^120 is exact.
__device__ __forceinline__ uint32_t widen2(uint32_t t) {
  const uint32_t y = ((t >> 4) & 0x07F007F0u) | (t & 0x80008000u);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(y), "r"(0x7B807B80u));
  return r;
}
// the 16 values of piece c (key c / 8, dims 16 (c % 8) ..) of a block to their place in the 16-bit tile
// [half][128 keys][64 dims]
__device__ __forceinline__ void store16(uint8_t* tile, int c, const uint32_t (&y)[8]) {
  const int key = c >> 3, d = (c & 7) * 16;
  uint8_t* base = tile + (d >> 6) * 16384;
  const uint32_t at0 = sw128_offset(key, (d & 63) * 2), at1 = sw128_offset(key, (d & 63) * 2 + 16);
  const uint4 lo = make_uint4(y[0], y[1], y[2], y[3]), hi = make_uint4(y[4], y[5], y[6], y[7]);
  // the lanes of the second dim half store in the other order: the halves' rows share banks
  const bool swap = d >= 64;
  *reinterpret_cast<uint4*>(base + (swap ? at1 : at0)) = swap ? hi : lo;
  *reinterpret_cast<uint4*>(base + (swap ? at0 : at1)) = swap ? lo : hi;
}
template <bool NANS>
__device__ __forceinline__ void widen16_bf16(uint8_t* tile, int c, const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = widen2(__byte_perm(w[i], 0, 0x1404));       // codes 0 and 1
    y[2 * i + 1] = widen2(__byte_perm(w[i], 0, 0x3424));   // codes 2 and 3
  }
  if (NANS) {                                              // the moved bits of a NaN code are 480: make them NaN
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((y[i] & 0x7FFFu) == 0x43F0u) y[i] |= 0x7FC0u;
      if ((y[i] & 0x7FFF0000u) == 0x43F00000u) y[i] |= 0x7FC00000u;
    }
  }
  store16(tile, c, y);
}
// V's values times 2^-15
__device__ __forceinline__ void widen16_f16(uint8_t* tile, int c, const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu)));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y[i]) : "r"(h), "r"(0x02000200u));   // exact: multiples of 2^-24, 4 bits
  }
  store16(tile, c, y);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// NaN into the dims of a partial (one head's, [16 pieces][16 heads][8 dims]) in which one of the first `keys` V rows has a NaN
// code.  Slow and rare: the codes once more, out of L2.
__device__ __forceinline__ void nan_dims(const uint8_t* v, int keys, __half* po) {
#pragma unroll 1
  for (int i = 0; i < keys * 8; ++i) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(v) + i);
    if (!has_nan(x)) continue;
#pragma unroll 1
    for (int b = 0; b < 16; ++b) {
      const uint32_t word = b < 8 ? (b < 4 ? x.x : x.y) : (b < 12 ? x.z : x.w);
      const int d = (i & 7) * 16 + b;
      if (((word >> (8 * (b & 3))) & 0x7Fu) == 0x7Fu) po[(d >> 3) * 128 + (d & 7)] = __ushort_as_half(0x7FFF);
    }
  }
}
// two fp32 operations an instruction (the same roundings)
__device__ __forceinline__ unsigned long long pair(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(unsigned long long v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Instruction descriptor, kind::f16: f16 x f16 -> fp32
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// ------------------------------------------------------------------ schedule
// An entry is a (row t, group g, slot) with a block; its bucket is (window of rows, sequence, g, block).  A window is
// 8192 rows: one group's queries of that many rows (32 MiB) stay in L2 while its blocks gather them again and again,
// those of 16,384 rows do not (the last 128K chunk 2.94 ms without windows, 2.84 with, 2.93 with 4096 rows).  Three
// kernels turn the entries into tiles of up to 8 of a bucket:
//   count  every entry's bucket and rank in it (a counter per bucket)
//   bases  every bucket's run of tiles, ceil(count / 8) of them, and its stretch of cost
//   place  every entry to tile base + rank / 8, place rank % 8; the first of a tile writes the tile's head, and the
//          tile as the first one of the CTAs whose share of the cost begins in it
// The counters' order decides which entries share a tile and where it stands, which no result depends on: an entry's
// rows of the products are its own.
struct SchedFp8Args {
  const int32_t* block_idx;   // [total_q][Hkv][topk]
  const int32_t* q_start;
  const int32_t* ctx_len;
  const int32_t* page_table;
  const float* k_scale;       // [pages][Hkv]
  const float* v_scale;
  unsigned long long* total;  // cost << 32 | number of tiles, zeroed with the counts behind it
  int* counts;                // [nbuckets]
  unsigned long long* bases;  // [nbuckets]: first cost << 32 | first tile
  int* starts;                // [ctas]: first tile of a CTA's share of the cost
  int2* entries;              // [total_q * Hkv * topk]: bucket (-1: none), rank
  int4* tile_rec;             // [max_tiles][4]: one 64-byte record per tile
  float2* part_lse;           // [total_q][Hkv][topk][16 heads], see AttnPrefillFp8Args
  int num_seqs, total_q, Hq, Hkv, topk, max_blocks, nbuckets, num_pages, max_tiles, cta_rows, ctas;
  int win_shift, win_buckets; // rows of a window (log2) and its buckets
};

// Blocks that most rows select (sink-like ones, each row's own block) would take thousands of atomics on one address, so
// a CTA first gathers its rows' entries per bucket in a shared-memory hash table and adds once per bucket.  Rows behind
// the last sequence have no entries; an entry whose block or page is out of range is recorded and left out (its partial
// gets lse = -inf).
constexpr int SCH8_HASH = 4096;                  // table slots: >= 2 x a CTA's entries when it is used
constexpr int SCH8_EPT = SCH8_HASH / 2 / 256;    // entries per thread (256 threads)

__global__ void __launch_bounds__(256) sched_fp8_count_kernel(const SchedFp8Args a) {
  __shared__ int s_key[SCH8_HASH];
  __shared__ int s_cnt[SCH8_HASH];               // entries per bucket, then the bucket's base
  pdl_launch_dependents();
  const int rows = min(a.total_q, __ldg(a.q_start + a.num_seqs));
  const int t0 = blockIdx.x * a.cta_rows;
  const int t1 = min(rows, t0 + a.cta_rows);
  if (t0 >= t1) return;
  const int per_row = a.Hkv * a.topk;
  const int nent = (t1 - t0) * per_row;
  const long e0 = static_cast<long>(t0) * per_row;
  auto bucket_of = [&](int el) -> int {
    const int b = __ldg(a.block_idx + e0 + el);
    if (b < 0) return -1;
    const int t = t0 + el / per_row, rem = el % per_row, g = rem / a.topk, slot = rem % a.topk;
    const int s = find_seq(a.q_start, a.num_seqs, t);
    const int p = __ldg(a.ctx_len + s) - __ldg(a.q_start + s + 1) + t;
    int page = -1;
    if (b < a.max_blocks && b * 128 <= p) page = __ldg(a.page_table + static_cast<long>(s) * a.max_blocks + b);
    if (page < 0 || page >= a.num_pages) {
      flag_error(MSA_DEV_BOUNDS);
      float2* pl = a.part_lse + ((static_cast<long>(t) * a.Hkv + g) * a.topk + slot) * ATTP_G;
      for (int h = 0; h < ATTP_G; ++h) pl[h] = make_float2(-INFINITY, 0.f);
      return -1;
    }
    return (t >> a.win_shift) * a.win_buckets + (s * a.Hkv + g) * a.max_blocks + b;
  };
  if (nent > SCH8_HASH / 2) {                     // rows too wide for the table: one atomic per entry
    for (int el = threadIdx.x; el < nent; el += blockDim.x) {
      const int bk = bucket_of(el);
      a.entries[e0 + el] = make_int2(bk, bk < 0 ? 0 : atomicAdd(&a.counts[bk], 1));
    }
    return;
  }
  for (int i = threadIdx.x; i < SCH8_HASH; i += blockDim.x) { s_key[i] = -1; s_cnt[i] = 0; }
  __syncthreads();
  int bks[SCH8_EPT], hs[SCH8_EPT], li[SCH8_EPT];
#pragma unroll
  for (int k = 0; k < SCH8_EPT; ++k) {
    const int el = threadIdx.x + k * 256;
    bks[k] = el < nent ? bucket_of(el) : -1;
  }
#pragma unroll
  for (int k = 0; k < SCH8_EPT; ++k) {
    hs[k] = -1;
    li[k] = 0;
    if (bks[k] < 0) continue;
    uint32_t h = (static_cast<uint32_t>(bks[k]) * 2654435761u) >> 20;   // 12 bits
    for (int probe = 0; probe < SCH8_HASH; ++probe) {                    // the table is at most half full
      const int prev = atomicCAS(&s_key[h], -1, bks[k]);
      if (prev == -1 || prev == bks[k]) { hs[k] = static_cast<int>(h); break; }
      h = (h + 1) & (SCH8_HASH - 1);
    }
    if (hs[k] >= 0) li[k] = atomicAdd(&s_cnt[hs[k]], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < SCH8_HASH; i += blockDim.x) {
    const int bk = s_key[i];
    if (bk >= 0) s_cnt[i] = atomicAdd(&a.counts[bk], s_cnt[i]);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < SCH8_EPT; ++k) {
    const int el = threadIdx.x + k * 256;
    if (el < nent) a.entries[e0 + el] = make_int2(bks[k], hs[k] >= 0 ? s_cnt[hs[k]] + li[k] : 0);
  }
}

// A tile's time is two units of cost; a change of bucket (its K to be widened, the pipeline to be filled again) is
// SCH8_CHANGE more.
constexpr int SCH8_CHANGE = 1;

// CTA = 1024 buckets, thread = 4: their exclusive sums of cost and tiles over the CTA, whose run begins where the totals
// stood.
__global__ void __launch_bounds__(256) sched_fp8_bases_kernel(const SchedFp8Args a) {
  __shared__ unsigned long long s_w[8], s_base;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  pdl_wait();
  const int i0 = (blockIdx.x * 256 + tid) * 4;
  unsigned long long tl[4], sum = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int n = i0 + k < a.nbuckets ? (a.counts[i0 + k] + ATTP_TOK - 1) / ATTP_TOK : 0;
    tl[k] = n ? static_cast<unsigned long long>(2 * n + SCH8_CHANGE) << 32 | n : 0ull;
    sum += tl[k];
  }
  unsigned long long v = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long n = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += n;
  }
  if (lane == 31) s_w[warp] = v;
  __syncthreads();
  if (tid == 0) {
    unsigned long long total = 0;
    for (int w = 0; w < 8; ++w) { const unsigned long long n = s_w[w]; s_w[w] = total; total += n; }
    s_base = total ? atomicAdd(a.total, total) : 0ull;
  }
  __syncthreads();
  unsigned long long at = s_base + s_w[warp] + v - sum;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (i0 + k < a.nbuckets) a.bases[i0 + k] = at;
    at += tl[k];
  }
}

// A tile's 64-byte record:
//   int[0] bucket, [1] first row of the block in the cache = (page * Hkv + g) * 128, [2] g, [3] b, [4] position offset of
//   the sequence (p = t + off), [5] entries n | tokens of the block that the sequence holds << 8, [6], [7] the block's K
//   and V scale, [8 .. 8+n) entries (t << 6 | slot), the rest of them whatever it was.
__global__ void __launch_bounds__(256) sched_fp8_place_kernel(const SchedFp8Args a) {
  pdl_launch_dependents();
  pdl_wait();
  const int per_row = a.Hkv * a.topk;
  const long e = static_cast<long>(blockIdx.x) * 256 + threadIdx.x;
  if (e >= static_cast<long>(min(a.total_q, __ldg(a.q_start + a.num_seqs))) * per_row) return;
  const int2 x = a.entries[e];
  if (x.x < 0) return;
  const int t = static_cast<int>(e / per_row), slot = static_cast<int>(e % a.topk);
  const unsigned long long base = a.bases[x.x];
  const int k = x.y / ATTP_TOK, tile = static_cast<int>(base & 0xFFFFFFFFu) + k, place = x.y % ATTP_TOK;
  int4* r = a.tile_rec + static_cast<long>(tile) * 4;
  reinterpret_cast<int*>(r + 2)[place] = (t << 6) | slot;
  if (place != 0) return;
  // CTA c's share begins at cost total c / ctas
  const unsigned long long total = *a.total >> 32, first = base >> 32;
  const unsigned long long from = k ? first + SCH8_CHANGE + 2 * k : first, to = first + SCH8_CHANGE + 2 * k + 2;
  const int c1 = static_cast<int>(min(static_cast<unsigned long long>(a.ctas), (to * a.ctas + total - 1) / total));
  for (int c = static_cast<int>((from * a.ctas + total - 1) / total); c < c1; ++c) a.starts[c] = tile;
  const int n = min(ATTP_TOK, a.counts[x.x] - x.y);
  const int y = x.x % a.win_buckets;
  const int b = y % a.max_blocks, g = (y / a.max_blocks) % a.Hkv, seq = y / (a.max_blocks * a.Hkv);
  const int page = __ldg(a.page_table + static_cast<long>(seq) * a.max_blocks + b);   // checked by the count
  const int row = page * a.Hkv + g, ctx = __ldg(a.ctx_len + seq);
  r[0] = make_int4(x.x, row * 128, g, b);
  r[1] = make_int4(ctx - __ldg(a.q_start + seq + 1), n | (min(128, ctx - b * 128) << 8),
                   __float_as_int(__ldg(a.k_scale + row)), __float_as_int(__ldg(a.v_scale + row)));
}

// ------------------------------------------------------------------ tiles
struct AttnPrefillFp8Args {
  const int4* tile_rec;      // [tiles][4] records written by sched_fp8_place_kernel
  const unsigned long long* total;   // cost << 32 | number of tiles
  const int* starts;         // [gridDim.x]
  const uint8_t* k_cache;    // [pages][Hkv][128][128] codes
  const uint8_t* v_cache;
  // Partials of (row, group, slot): O is not divided by l and counts codes, as f16 (bf16 would cost no less and take the error
  // against 64 bits from 1.7e-3, that of the output's own rounding, to 2.3e-3; f16's least step adds at most 2^-24 v_scale, 2^-15
  // of the least code), [16 pieces of 8 dims][16 heads][8], so that a
  // warp's stores are whole lines; of each head log2(sum) and v_scale / sum, the factor that O still wants.
  __half* part_o;            // [total_q][Hkv][topk][2048]
  float2* part_lse;          // [total_q][Hkv][topk][16 heads]
  int Hq, Hkv, topk;
  float scale_log2;
};

__global__ void __launch_bounds__(ATP8_THREADS, 1)
attn_prefill_fp8_kernel(const __grid_constant__ CUtensorMap tmap_q,     // q as [total_q*Hq][128]
                        const AttnPrefillFp8Args a) {
  extern __shared__ __align__(1024) uint8_t dsmem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = smem;                                  // 3 x 32 KiB: [half][128 rows][64]
  uint8_t* k_s = q_s + ATP8_QBUF * ATTP_QBYTES;         // 2 x: [half][128 keys][64]
  uint8_t* v_s = k_s + 2 * ATTP_KVBYTES;                // 2 x: [half][128 keys][64]

  // Per warpgroup w (its own tile sequence, so a parity never runs two phases ahead): s_full[w] S is in
  // TMEM, p_full[w] P is in TMEM (one arrival per warp), o_full[w] O[w] holds its tile, o_empty[w] O[w]
  // has been read (one arrival per warp).  k_full, v_full: a bucket's tile is widened (one arrival per converter
  // warp); k_empty, v_empty: its last S, its last P V is done.  K and V have two buffers each: a bucket's first S comes two
  // tiles before the last P V of the bucket before it, and with one buffer every change of bucket held P V up by 2,000
  // clocks.
  __shared__ uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], q_full[ATP8_QBUF], q_empty[ATP8_QBUF], s_full[2],
      p_full[2], o_full[2], o_empty[2], rec_full[ATP8_RECS], drain_bar[2];
  __shared__ int4 s_rec[ATP8_RECS][4];            // the softmax warps' records (the first field: which bucket of this CTA's)
  __shared__ __align__(16) int s_vnan[4][4];      // per bucket (a ring) and converter warp: its first V row with a NaN code, or 128
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 4);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 4);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < ATP8_QBUF; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_empty[i], 4);
    }
    for (int i = 0; i < ATP8_RECS; ++i) mbar_init(&rec_full[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&drain_bar[i], 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  pdl_wait();                                            // the records
  // Tiles come by bucket.  All CTAs move through the list together, ATP8_RUN tiles each and round, so that they gather
  // from the same window and group.  A short list is cut into one run per CTA instead, so that a bucket's tiles stay
  // together (runs of 32: mixed chunks 302 us instead of 269), at equal shares of the cost (equal numbers of tiles left
  // the SMs idle for a quarter of the time).
  const int T = static_cast<int>(*a.total & 0xFFFFFFFFu);
  const int G = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
  const bool shortlist = T <= 2 * G * ATP8_RUN;
  const int full = T / (G * ATP8_RUN);                      // whole rounds
  const int start = shortlist ? (T ? a.starts[c] : 0) : c * ATP8_RUN;
  const int ntile = shortlist ? (T ? (c + 1 < G ? a.starts[c + 1] : T) - start : 0)
                              : full * ATP8_RUN + max(0, min(ATP8_RUN, T - full * G * ATP8_RUN - start));
  // global tile of this CTA's i-th tile
  auto tile_of = [=](int i) -> int { return shortlist ? start + i : (i / ATP8_RUN) * (G * ATP8_RUN) + start + i % ATP8_RUN; };

  if (warp < 4) {
  regs_dec<ATP8_REGS_CTRL>();
  if (warp == 0) {
    // ------------------------------------------------------------ producer warp
    // Tile records arrive 32 at a time (one per lane, a single coalesced load), so no record
    // fetch sits on the issue path; lanes 0..15 issue the tile's query-row copies in parallel.
    if (lane == 0) tma_prefetch_desc(&tmap_q);
    uint32_t q_used = 0, q_parity_bits = 0;   // lane 0: per query buffer, issued at least once / parity of the last issue
    // A group's query rows are gathered again by every block they selected: keep them in L2.
    const uint64_t pol_q = l2_policy_evict_last();
    int4 ra = make_int4(-1, 0, 0, 0), rb = make_int4(0, 0, 0, 0), rc = rb, rd = rb;   // record of tile (batch + lane)
    int cur = -1, nbucket = -1;
    for (int i = 0; i < ntile; ++i) {
      if (__any_sync(0xFFFFFFFFu, s_abort != 0)) break;
      if ((i & 31) == 0 && i + lane < ntile) {
        const int4* p = a.tile_rec + static_cast<long>(tile_of(i + lane)) * 4;
        ra = __ldg(p); rb = __ldg(p + 1); rc = __ldg(p + 2); rd = __ldg(p + 3);
      }
      const int src = i & 31;
      const int g = __shfl_sync(0xFFFFFFFFu, ra.z, src);
      const int n = __shfl_sync(0xFFFFFFFFu, rb.y, src) & 15;
      // the tile's entries (t << 6 | slot)
      const int e0 = __shfl_sync(0xFFFFFFFFu, rc.x, src), e1 = __shfl_sync(0xFFFFFFFFu, rc.y, src);
      const int e2 = __shfl_sync(0xFFFFFFFFu, rc.z, src), e3 = __shfl_sync(0xFFFFFFFFu, rc.w, src);
      const int e4 = __shfl_sync(0xFFFFFFFFu, rd.x, src), e5 = __shfl_sync(0xFFFFFFFFu, rd.y, src);
      const int e6 = __shfl_sync(0xFFFFFFFFu, rd.z, src), e7 = __shfl_sync(0xFFFFFFFFu, rd.w, src);
      bool ok = true;
      const int qb = i % ATP8_QBUF;
      const uint32_t qpar = static_cast<uint32_t>((i / ATP8_QBUF) & 1);
      if (lane == 0) {
        ok = mbar_wait(&q_empty[qb], qpar ^ 1u, &s_abort);
        if (ok) {
          mbar_arrive_expect_tx(&q_full[qb], n * 4096);
          q_used |= 1u << qb;
          q_parity_bits = (q_parity_bits & ~(1u << qb)) | (qpar << qb);
        }
      }
      if (!__shfl_sync(0xFFFFFFFFu, ok ? 1 : 0, 0)) break;
      // S(i-3) is done, so P(i-5) was written and tile i-7 is over: its record may go
      const int bucket = __shfl_sync(0xFFFFFFFFu, ra.x, src);
      if (bucket != cur) { ++nbucket; cur = bucket; }
      if (lane == src) {
        int4* rec = s_rec[i % ATP8_RECS];
        rec[0] = make_int4(nbucket, ra.y, ra.z, ra.w);
        rec[1] = rb;
        rec[2] = rc;
        rec[3] = rd;
        mbar_arrive(&rec_full[i % ATP8_RECS]);
      }
      __syncwarp();
      // query rows of the tile's entries (MMA row 16e + head), [half][128 rows][64 dims] swizzled:
      // lane 2e + half issues entry e's half
      {
        const int el = lane >> 1, half = lane & 1;
        const int en = el == 0 ? e0 : el == 1 ? e1 : el == 2 ? e2 : el == 3 ? e3 : el == 4 ? e4 : el == 5 ? e5
                     : el == 6 ? e6 : e7;
        if (lane < 2 * ATTP_TOK && el < n)
          tma_load_2d_hint(q_s + qb * ATTP_QBYTES + half * 16384 + el * 2048, &tmap_q, &q_full[qb], half * 64,
                           (en >> 6) * a.Hq + g * ATTP_G, pol_q);
      }
    }
    if (lane == 0 && s_abort) {                  // let issued copies land before the CTA exits
      for (int j = 0; j < ATP8_QBUF; ++j)
        if (q_used & (1u << j)) mbar_wait_drain(&q_full[j], (q_parity_bits >> j) & 1u);
    }
  } else if (warp == 1) {
   if (lane == 0) {
    // ------------------------------------------------------------ S issuer
    // Tile i: S(i) = Q K^T into S[i % 2] (A and B from shared memory).  S(i) overwrites the columns that P V(i-2) reads.
    // One thread's instruction latency is on the critical path: descriptors are built once (only the 14-bit start
    // address, in 16-byte units, moves) and ring positions are counters.
    const uint32_t id_s = idesc_bf16(128, 128, false, false);
    const uint64_t qdesc0 = sdesc_sw128(smem_u32(q_s), 16, 1024);
    const uint64_t kdesc0 = sdesc_sw128(smem_u32(k_s), 16, 1024);
    uint64_t kdesc = kdesc0;
    int qb = 0;
    uint32_t qph = 0;
    int cur_bucket = -1;
    uint32_t kvit = 0;
    int nbucket = ntile > 0 ? __ldg(&a.tile_rec[static_cast<long>(tile_of(0)) * 4].x) : -1;
    for (int i = 0; i < ntile && !s_abort; ++i) {
      const int bucket = nbucket;
      if (i + 1 < ntile) nbucket = __ldg(&a.tile_rec[static_cast<long>(tile_of(i + 1)) * 4].x);
      if (bucket != cur_bucket) {
        if (cur_bucket >= 0) umma_commit(&k_empty[(kvit & 1) ^ 1]);   // the previous bucket's last S is issued
        if (!mbar_wait(&k_full[kvit & 1], (kvit >> 1) & 1, &s_abort)) break;
        kdesc = kdesc0 + static_cast<uint64_t>((kvit & 1) * (ATTP_KVBYTES >> 4));
        ++kvit;
        cur_bucket = bucket;
      }
      const int sb = i & 1;
      if (!mbar_wait(&q_full[qb], qph, &s_abort)) break;
      if (i >= 2 && !mbar_wait(&o_full[sb], static_cast<uint32_t>((i >> 1) - 1) & 1u, &s_abort)) break;   // P V(i-2)
      tc_fence_after();
      const uint32_t d = tmem + ATTP_TM_S + sb * 128;
      const uint64_t qd = qdesc0 + static_cast<uint64_t>((qb * ATTP_QBYTES) >> 4);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {   // 16 dims per step: 32 bytes within a 128-byte row, halves 16 KiB apart
        const uint32_t off16 = (kk >> 2) * 1024 + (kk & 3) * 2;
        umma_bf16_ss(d, qd + off16, kdesc + off16, id_s, kk > 0 ? 1u : 0u);
      }
      umma_commit(&s_full[sb]);
      umma_commit(&q_empty[qb]);
      if (++qb == ATP8_QBUF) { qb = 0; qph ^= 1u; }
    }
    if (s_abort) {
      umma_commit(&drain_bar[0]);
      mbar_wait_drain(&drain_bar[0], 0);
    }
   }
  } else if (warp == 2) {
   if (lane == 0) {
    // ------------------------------------------------------------ P V issuer
    // O[i % 2] = P(i) V, P(i) read from TMEM over the first half of S[i % 2].
    const uint32_t id_pv = idesc_f16(128, 128, true);
    const uint64_t vdesc0 = sdesc_sw128(smem_u32(v_s), 16384, 1024);
    uint32_t vit = 0;
    bool v_wait = true;
    int bucket = ntile > 0 ? __ldg(&a.tile_rec[static_cast<long>(tile_of(0)) * 4].x) : -1;
    for (int i = 0; i < ntile && !s_abort; ++i) {
      const int next = i + 1 < ntile ? __ldg(&a.tile_rec[static_cast<long>(tile_of(i + 1)) * 4].x) : -1;
      const int pb = i & 1;
      const uint32_t ph = static_cast<uint32_t>((i >> 1) & 1);
      if (v_wait && !mbar_wait(&v_full[vit & 1], (vit >> 1) & 1, &s_abort)) break;
      v_wait = false;
      if (!mbar_wait(&o_empty[pb], ph ^ 1u, &s_abort)) break;   // tile i-2's O has been read
      if (!mbar_wait(&p_full[pb], ph, &s_abort)) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)   // 16 keys per step: 2048 bytes of V rows
        umma_bf16_ts(tmem + ATTP_TM_O + pb * 128, tmem + ATTP_TM_S + pb * 128 + kk * 8,
                     vdesc0 + static_cast<uint64_t>((vit & 1) * (ATTP_KVBYTES >> 4)) + 128 * kk, id_pv,
                     kk > 0 ? 1u : 0u);
      umma_commit(&o_full[pb]);
      if (next != bucket) {              // the last of its bucket
        umma_commit(&v_empty[vit & 1]);
        ++vit;
        v_wait = true;
        bucket = next;
      }
    }
    if (s_abort) {
      umma_commit(&drain_bar[1]);
      mbar_wait_drain(&drain_bar[1], 0);
    }
   }
  }
  } else if (warp < 8) {
    regs_dec<ATP8_REGS_CONV>();
    // ------------------------------------------------------------ converters: a bucket's codes to 16 bits
    // A thread takes every 128th 16-byte piece of the tile.  Its buffers are free when the last S and the last P V of
    // the bucket before the previous one are done, so that a bucket is widened while the previous one's tiles run.
    const int ct = tid - 128;
    int4 ra = make_int4(-1, 0, 0, 0), rb = ra;               // records of tiles (batch + lane)
    int i = 0, cur = -1, row = 0, valid = 0;
    auto next_bucket = [&]() -> bool {                       // to the next bucket of this CTA's tiles; uniform
      while (i < ntile) {
        const int at = i & 31;
        if (at == 0 && i + lane < ntile) {
          const int4* p = a.tile_rec + static_cast<long>(tile_of(i + lane)) * 4;
          ra = __ldg(p);
          rb = __ldg(p + 1);
        }
        // lanes of this batch's tiles from i on whose bucket is another one
        const uint32_t others = __ballot_sync(0xFFFFFFFFu, ra.x != cur && i - at + lane < ntile) & (0xFFFFFFFFu << at);
        if (others) {
          const int src = __ffs(others) - 1;
          cur = __shfl_sync(0xFFFFFFFFu, ra.x, src);
          row = __shfl_sync(0xFFFFFFFFu, ra.y, src);
          valid = __shfl_sync(0xFFFFFFFFu, rb.y, src) >> 8;
          i += src - at + 1;
          return true;
        }
        i += 32 - at;
      }
      return false;
    };
    uint4 x[8];
    auto codes = [&](const uint8_t* cache) { return reinterpret_cast<const uint4*>(cache + static_cast<long>(row) * 128) + ct; };
    auto load = [&](const uint8_t* cache) {
      const uint4* p = codes(cache);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = __ldg(p + k * 128);
    };
    // V comes by way of L2: it is wanted soon after K, and from DRAM, beside the partials' stores, a change of bucket
    // waited up to 12 us for it.
    auto prefetch_v = [&]() {
      asm volatile("prefetch.global.L2::evict_last [%0];" ::"l"(a.v_cache + (static_cast<long>(row) + ct) * 128));
    };
    bool have = next_bucket(), ok = true;
    if (have) {
      load(a.k_cache);
      prefetch_v();
    }
    for (uint32_t it = 0; have && ok; ++it) {
      const bool nans = warp_has_nan(x);
      ok = mbar_wait_warp(&k_empty[it & 1], ((it >> 1) & 1) ^ 1, &s_abort);
      if (!ok) break;
      if (nans) {                     // rare: piece by piece, out of L2 again
#pragma unroll 1
        for (int k = 0; k < 8; ++k) widen16_bf16<true>(k_s + (it & 1) * ATTP_KVBYTES, k * 128 + ct, __ldg(codes(a.k_cache) + k * 128));
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) widen16_bf16<false>(k_s + (it & 1) * ATTP_KVBYTES, k * 128 + ct, x[k]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[it & 1]);
      load(a.v_cache);
      ok = mbar_wait_warp(&v_empty[it & 1], ((it >> 1) & 1) ^ 1, &s_abort);
      if (!ok) break;
      int bad = 128;
      if (valid < 128 || warp_has_nan(x)) {
        // slots behind the sequence hold anything; a NaN that counts is noted and taken out (0 x NaN is NaN for the
        // rows that do not see it)
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
          const int key = (k * 128 + ct) >> 3;
          uint4 y = make_uint4(0u, 0u, 0u, 0u);
          if (key < valid) y = __ldg(codes(a.v_cache) + k * 128);
          if (has_nan(y)) {
            bad = min(bad, key);
            y = without_nan(y);
          }
          widen16_f16(v_s + (it & 1) * ATTP_KVBYTES, k * 128 + ct, y);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) widen16_f16(v_s + (it & 1) * ATTP_KVBYTES, k * 128 + ct, x[k]);
      }
      bad = __reduce_min_sync(0xFFFFFFFFu, bad);
      if (lane == 0) s_vnan[it & 3][warp - 4] = bad;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[it & 1]);
      have = next_bucket();
      if (have) {
        load(a.k_cache);
        prefetch_v();
      }
    }
  } else {
    regs_inc<ATP8_REGS_SOFTMAX>();
    // ------------------------------------------------------------ two softmax + epilogue warpgroups
    // Warpgroup w takes the CTA's tiles i = w, w + 2, ...; it owns S[w], P[w] and O[w].
    // Every warp runs on its own (its 32 TMEM lanes = 2 entries x 16 heads): it waits, arrives and
    // stores its rows without waiting for the other warps.
    const int w = (warp - 8) >> 2;
    const int quarter = warp & 3;                 // TMEM lanes 32*quarter .. +31
    const int r = quarter * 32 + lane;            // MMA row = entry * 16 + head
    const int e = r >> 4, h = r & 15;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int nj = (ntile - w + 1) / 2;
    int4 h0 = make_int4(0, 0, 0, 0), h1 = h0;      // the record of tile j, and this row's entry
    int ent = 0;
    auto next_record = [&](int i) -> bool {
      if (!mbar_wait_warp(&rec_full[i % ATP8_RECS], static_cast<uint32_t>((i / ATP8_RECS) & 1), &s_abort)) return false;
      const int4* rec = s_rec[i % ATP8_RECS];
      h0 = rec[0];
      h1 = rec[1];
      ent = reinterpret_cast<const int*>(rec + 2)[e];
      return true;
    };
    bool ok = nj == 0 || next_record(w);
    for (int j = 0; j < nj && ok; ++j) {         // exit decisions are uniform over the warp
      const int nbucket = h0.x, n = h1.y & 15;
      const float ks = __int_as_float(h1.z), vs = __int_as_float(h1.w);
      const float sa = a.scale_log2 * fabsf(ks);
      const float sc = sa < 1e-36f ? 1e-36f : sa;   // not 0: the masked -inf * 0 is NaN; a NaN scale stays NaN
      const bool valid = e < n;
      const int t = ent >> 6;
      const long part = (static_cast<long>(t) * a.Hkv + h0.z) * a.topk + (ent & 63);
      const int vis = valid ? min(128, t + h1.x - h0.w * 128 + 1) : 128;  // visible keys of the block

      // ---- S = Q K^T is in TMEM: the row's 128 scores in registers, max over the visible keys
      if (!mbar_wait_warp(&s_full[w], static_cast<uint32_t>(j & 1), &s_abort)) break;
      tc_fence_after();
      const uint32_t s_addr = lane_addr + ATTP_TM_S + w * 128;
      float v0[32], v1[32], v2[32], v3[32];
      tmem_ld32(s_addr, v0);
      tmem_ld32(s_addr + 32, v1);
      tmem_ld32(s_addr + 64, v2);
      tmem_ld32(s_addr + 96, v3);
      tmem_ld_wait();
      if (ks < 0.f) {                         // a negative scale: the scores' order is that of -S
#pragma unroll
        for (int c = 0; c < 32; ++c) { v0[c] = -v0[c]; v1[c] = -v1[c]; v2[c] = -v2[c]; v3[c] = -v3[c]; }
      }
      if (vis < 128) {                            // the query's own block: keys after it do not count
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          if (c >= vis) v0[c] = -INFINITY;
          if (32 + c >= vis) v1[c] = -INFINITY;
          if (64 + c >= vis) v2[c] = -INFINITY;
          if (96 + c >= vis) v3[c] = -INFINITY;
        }
      }
      float mx[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) mx[q] = -INFINITY;
#pragma unroll
      for (int c = 0; c < 32; ++c) mx[c & 7] = fmax3(mx[c & 7], fmaxf(v0[c], v1[c]), fmaxf(v2[c], v3[c]));
      const float m = fmaxf(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], fmax3(mx[4], mx[5], mx[6]), mx[7]));
      // P at most 2^14: with V's 2^-15 that is 1/2, so that a sum of 128 codes of 448 stays an f16 number with room for the
      // rounding of m sc; -inf only on rows past the tile's entries
      const float mc = (m > -INFINITY) ? fmaf(m, sc, -14.f) : 0.f;
      float off = mc;
      if (fabsf(mc) >= 65536.f) {                 // huge scores: that rounding would be whole powers of two, so m goes first
        off = -14.f;
#pragma unroll
        for (int c = 0; c < 32; ++c) { v0[c] -= m; v1[c] -= m; v2[c] -= m; v3[c] -= m; }
      }
      // ---- P = exp2(scale * S - max) as f16 pairs into P[w] (TMEM), two halves of 64 keys
      float l0 = 0.f, l1 = 0.f;
      const unsigned long long sc2 = pair(sc, sc), mc2 = pair(-off, -off);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t pk[32];
#pragma unroll
        for (int q2 = 0; q2 < 32; ++q2) {
          const int c = half * 64 + q2 * 2;
          const float x0 = c < 32 ? v0[c] : c < 64 ? v1[c - 32] : c < 96 ? v2[c - 64] : v3[c - 96];
          const float x1 = c + 1 < 32 ? v0[c + 1] : c + 1 < 64 ? v1[c - 31] : c + 1 < 96 ? v2[c - 63] : v3[c - 95];
          float p0, p1;
          unpair(fma2(pair(x0, x1), sc2, mc2), p0, p1);
          p0 = exp2f(p0);                          // exp2(-inf) = 0
          p1 = exp2f(p1);
          if (q2 & 1) l1 += p0 + p1; else l0 += p0 + p1;
          pk[q2] = pack_f16(p0, p1);
        }
        tmem_st32(lane_addr + ATTP_TM_S + w * 128 + half * 32, pk);   // S columns already in registers
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[w]);
      // ---- while the tensor cores multiply: the row's statistics, the next record
      const float l = l0 + l1;
      if (j + 1 < nj) ok = next_record(2 * j + 2 + w);

      // ---- O = P V is in TMEM: read it, release the accumulator, O as f16 to its partial
      if (!mbar_wait_warp(&o_full[w], static_cast<uint32_t>(j & 1), &s_abort)) break;
      tc_fence_after();
      float o0[32], o1[32], o2[32], o3[32];
      const uint32_t o_addr = lane_addr + ATTP_TM_O + w * 128;
      tmem_ld32(o_addr, o0);
      tmem_ld32(o_addr + 32, o1);
      tmem_ld32(o_addr + 64, o2);
      tmem_ld32(o_addr + 96, o3);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[w]);
      if (valid) {
        uint4* po = reinterpret_cast<uint4*>(a.part_o + part * 2048) + h;
#pragma unroll
        for (int c = 0; c < 16; ++c) {            // output dims 8c .. 8c+7
          const float* ov = c < 4 ? o0 + c * 8 : c < 8 ? o1 + c * 8 - 32 : c < 12 ? o2 + c * 8 - 64 : o3 + c * 8 - 96;
          __stcs(po + c * 16, make_uint4(pack_f16(ov[0], ov[1]), pack_f16(ov[2], ov[3]), pack_f16(ov[4], ov[5]),
                                         pack_f16(ov[6], ov[7])));
        }
      }
      if (valid) {
        // NaN codes among the V rows that this row sees (the converters took them out): NaN in their dims
        const int4 vn = *reinterpret_cast<const int4*>(s_vnan[nbucket & 3]);
        if (min(min(vn.x, vn.y), min(vn.z, vn.w)) < vis) {
          // this tile's record is still there: tile i + 8's needs this warp's P of tile i + 2
          const int row = s_rec[(2 * j + w) % ATP8_RECS][0].y;
          nan_dims(a.v_cache + static_cast<long>(row) * 128, vis, a.part_o + part * 2048 + h * 8);
        }
        a.part_lse[part * ATTP_G + h] = make_float2(mc + log2f(l), vs / (l * 0x1p-15f));
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ merge
struct MergeFp8Args {
  const __half* part_o;          // [total_q][Hkv][topk][2048], as the tiles' kernel leaves them
  const float2* part_lse;        // [total_q][Hkv][topk][16 heads]
  const int32_t* block_idx;      // [total_q][Hkv][topk]
  const int32_t* q_start;
  __nv_bfloat16* out;            // [total_q][Hq][128]
  float* lse;                    // [total_q][Hq] or null
  int num_seqs, Hq, Hkv, topk;
};

// out = sum_b w_b O_b, w_b = 2^(lse_b - max) (v_scale / l)_b / sum 2^(lse - max), over the partials of a row and group.
// One CTA per (row, group): 16 heads x 16 threads x 8 output dims, every load of four slots issued before the first is
// used, six CTAs an SM (eight slots and four CTAs: 2,048 rows of one group 45.8 us instead of 44.6, the rest alike).  Rows
// behind the last sequence are left as they were, slots without a partial (not selected, or lse = -inf) count nothing, a
// NaN gets through.
__global__ void __launch_bounds__(256, 6) attn_merge_fp8_kernel(const MergeFp8Args a) {
  __shared__ float s_l[MRG_MAXK][ATTP_G], s_f[MRG_MAXK][ATTP_G];
  const int t = blockIdx.x / a.Hkv, g = blockIdx.x % a.Hkv;
  if (t >= __ldg(a.q_start + a.num_seqs)) return;
  const int h = threadIdx.x & 15, d8 = threadIdx.x >> 4;
  const int head = g * ATTP_G + h;
  const long first = static_cast<long>(blockIdx.x) * a.topk;            // of the row and group's slots
  const uint4* po = reinterpret_cast<const uint4*>(a.part_o) + first * 256 + threadIdx.x;
  for (int s = d8; s < a.topk; s += 16) {
    float2 v = make_float2(-INFINITY, 0.f);
    if (__ldg(a.block_idx + first + s) >= 0) v = __ldg(a.part_lse + first * ATTP_G + s * ATTP_G + h);
    s_l[s][h] = v.x;
    s_f[s][h] = v.y;
  }
  __syncthreads();
  float mx = -3e38f;                        // finite: a row of NaN partials stays NaN
  for (int s = 0; s < a.topk; ++s) mx = fmaxf(mx, s_l[s][h]);
  float wsum = 0.f;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  // 4 slots per round, every partial load of the round issued before the first is used
  for (int s0 = 0; s0 < a.topk; s0 += 4) {
    uint4 o[4];
    float w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = s0 + k;
      w[k] = s < a.topk ? s_l[s][h] : -INFINITY;
      o[k] = w[k] != -INFINITY ? __ldcs(po + static_cast<long>(s) * 256) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (w[k] == -INFINITY) continue;
      const float e = exp2f(w[k] - mx), f = e * s_f[s0 + k][h];
      wsum += e;
      float2 v;
      v = __half22float2(*reinterpret_cast<const __half2*>(&o[k].x)); acc[0] = fmaf(f, v.x, acc[0]); acc[1] = fmaf(f, v.y, acc[1]);
      v = __half22float2(*reinterpret_cast<const __half2*>(&o[k].y)); acc[2] = fmaf(f, v.x, acc[2]); acc[3] = fmaf(f, v.y, acc[3]);
      v = __half22float2(*reinterpret_cast<const __half2*>(&o[k].z)); acc[4] = fmaf(f, v.x, acc[4]); acc[5] = fmaf(f, v.y, acc[5]);
      v = __half22float2(*reinterpret_cast<const __half2*>(&o[k].w)); acc[6] = fmaf(f, v.x, acc[6]); acc[7] = fmaf(f, v.y, acc[7]);
    }
  }
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
  uint4 r;
  r.x = pack_bf16(acc[0] * inv, acc[1] * inv);
  r.y = pack_bf16(acc[2] * inv, acc[3] * inv);
  r.z = pack_bf16(acc[4] * inv, acc[5] * inv);
  r.w = pack_bf16(acc[6] * inv, acc[7] * inv);
  *reinterpret_cast<uint4*>(a.out + (static_cast<long>(t) * a.Hq + head) * 128 + d8 * 8) = r;
  if (a.lse && d8 == 0)
    a.lse[static_cast<long>(t) * a.Hq + head] = wsum == 0.f ? -INFINITY : (mx + log2f(wsum)) * 0.69314718055994531f;
}

}  // namespace msa
