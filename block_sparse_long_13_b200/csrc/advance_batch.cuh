// msa_advance_batch: the index arrays of a step from the requests' token counts, on the device.
//
// Sequence s holds ctx_len[s] tokens in ceil(ctx_len[s] / 128) pages.  delta[s] > 0 appends that many tokens
// (this step's query rows), delta[s] < 0 takes tokens back (rejected drafts; -ctx_len[s] ends the request).
//   after[s]   = ctx_len[s] + delta[s],  have = ceil(ctx_len / 128),  want = ceil(after / 128)
//   q_start    = exclusive sum of max(delta, 0)
//   grow / back = max(0, want - have) / max(0, have - want) pages; their exclusive sums G, B
//   page_table[s][have + j] = ring[(head + G[s] + j) mod P]                  (pages leave at the ring's head)
//   ring[(head + count + B[s] + j) mod P] = page_table[s][want + j]          (and come back at its tail)
//   slot_map[q_start[s] + i] = page * 128 + offset of position ctx_len[s] + i
// Pages given back in a call are not taken in the same call, so the ring's reads and writes are disjoint; so
// are the page table's (a sequence either grows or shrinks).  The order is that of (sequence, block): the
// result does not depend on timing.  All or nothing: a call whose pages or arguments do not fit changes no
// length, page or ring entry.
//
// A few KiB to a few MiB move; the sums' latency bounds it.  One CTA scans the sequences 1024 at a time into shared
// memory, then every thread takes pages and rows by binary search in the sums.  A slot map of more than ADV_ONE rows
// is left to a second kernel of many CTAs, which needs no more than the finished q_start, ctx_len and page_table
// (448,000 rows of 1024 prompts: in the one CTA 364 us, in a cluster of eight 36 us, so 12.6 us).
#pragma once
#include "common.cuh"
#include "launch_order.cuh"

namespace msa {

constexpr int ADV_THREADS = 1024;
constexpr int ADV_MAXSEQ = 8192;
constexpr int ADV_ONE = 8192;          // rows of a slot map that the one CTA writes
constexpr int SLOT_THREADS = 512, SLOT_ROWS = 4;   // rows of a thread and round

struct AdvanceArgs {
  const int32_t* delta;
  const int32_t* ctx_len;
  int32_t* page_table;           // [num_seqs][max_blocks]
  int32_t* ring;                 // [num_pages]
  const int32_t* pool;           // head, count, -, -
  int32_t* ctx_out;              // ctx_len itself or disjoint
  int32_t* pool_out;             // pool itself or disjoint
  int32_t* q_start;              // [num_seqs + 1]
  int32_t* slot_map;             // [max_rows] or null
  int num_seqs, max_blocks, num_pages, max_rows;
};

__host__ __device__ constexpr int advance_smem(int num_seqs) { return (4 * num_seqs + 3) * 4; }

// largest s < n with sum[s] <= x
__device__ __forceinline__ int adv_find(const int* sum, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sum[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ unsigned long long warp_scan(unsigned long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long n = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

__global__ void __launch_bounds__(ADV_THREADS) advance_batch_kernel(const AdvanceArgs a) {
  extern __shared__ int adv_smem[];
  const int n = a.num_seqs;
  int* s_old = adv_smem;             // [n] tokens before
  int* s_q = s_old + n;              // [n + 1] row sums
  int* s_g = s_q + n + 1;            // [n + 1] page sums: grow
  int* s_b = s_g + n + 1;            // [n + 1] and back
  __shared__ unsigned long long w_rows[32], w_pages[32], c_rows, c_pages;
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  const bool maps = a.slot_map && a.max_rows <= ADV_ONE;
  const int head = a.pool[0], count = a.pool[1], P = a.num_pages;
  if (tid == 0) {
    c_rows = c_pages = 0;
    s_bad = head < 0 || head >= P || count < 0 || count > P;
  }
  __syncthreads();
  for (int base = 0; base < n; base += ADV_THREADS) {
    const int s = base + tid;
    unsigned long long rows = 0, pages = 0;          // pages: back << 32 | grow
    if (s < n) {
      const int old = a.ctx_len[s];
      const long after = static_cast<long>(old) + a.delta[s];
      s_old[s] = old;
      if (old < 0 || after < 0 || old > static_cast<long>(a.max_blocks) * 128 || after > static_cast<long>(a.max_blocks) * 128) {
        s_bad = 1;
      } else {
        const int have = static_cast<int>((static_cast<long>(old) + 127) >> 7), want = static_cast<int>((after + 127) >> 7);
        rows = after > old ? after - old : 0;
        pages = want > have ? static_cast<unsigned>(want - have) : static_cast<unsigned long long>(have - want) << 32;
      }
    }
    const unsigned long long r = warp_scan(rows, lane), g = warp_scan(pages, lane);
    if (lane == 31) { w_rows[warp] = r; w_pages[warp] = g; }
    __syncthreads();
    if (warp == 0) {
      w_rows[lane] = warp_scan(w_rows[lane], lane);
      w_pages[lane] = warp_scan(w_pages[lane], lane);
    }
    __syncthreads();
    const unsigned long long er = c_rows + (warp ? w_rows[warp - 1] : 0) + r - rows;
    const unsigned long long eg = c_pages + (warp ? w_pages[warp - 1] : 0) + g - pages;
    if (s < n) {
      s_q[s] = static_cast<int>(er);                 // sums past 2^31 are refused below
      s_g[s] = static_cast<int>(eg & 0xFFFFFFFFu);
      s_b[s] = static_cast<int>(eg >> 32);
    }
    __syncthreads();
    if (tid == 0) { c_rows += w_rows[31]; c_pages += w_pages[31]; }
    __syncthreads();
  }
  const unsigned long long rows_l = c_rows;
  const long need_l = static_cast<long>(c_pages & 0xFFFFFFFFu), free_l = static_cast<long>(c_pages >> 32);
  // counts of pages are at most max_seqs * max_blocks = 2^27, so the packed halves cannot run over
  const bool bad = s_bad || rows_l > 0x7FFFFFFFull || (a.slot_map && rows_l > static_cast<unsigned long long>(a.max_rows)) ||
                   count + free_l > P;
  const int missing = bad ? -1 : static_cast<int>(need_l > count ? need_l - count : 0);
  const bool ok = missing == 0;
  const int need = static_cast<int>(need_l), freed = static_cast<int>(free_l), rows = static_cast<int>(rows_l);
  if (tid == 0) {
    if (bad) flag_error(MSA_DEV_BOUNDS);
    s_q[n] = rows; s_g[n] = need; s_b[n] = freed;
    const int h = head + need;
    a.pool_out[0] = ok ? (h >= P ? h - P : h) : head;
    a.pool_out[1] = ok ? count - need + freed : count;
    a.pool_out[2] = missing;
    a.pool_out[3] = ok ? rows : 0;
  }
  __syncthreads();
  for (int s = tid; s <= n; s += ADV_THREADS) {
    if (s < n) a.ctx_out[s] = ok ? s_old[s] + a.delta[s] : s_old[s];
    a.q_start[s] = ok ? s_q[s] : 0;
  }
  const int filled = ok ? rows : 0;
  if (maps)
    for (int r = filled + tid; r < a.max_rows; r += ADV_THREADS) a.slot_map[r] = -1;
  if (!ok) return;
  auto wrap = [P](int i) { return i >= P ? i - P : i; };
  auto checked = [P](int page) {
    const bool fine = page >= 0 && page < P;
    if (!fine) flag_error(MSA_DEV_BOUNDS);
    return fine ? page : -1;
  };
  for (int i = tid; i < freed; i += ADV_THREADS) {
    const int s = adv_find(s_b, n, i);
    const int want = (s_old[s] + a.delta[s] + 127) >> 7;
    a.ring[wrap(wrap(head + count) + i)] = checked(a.page_table[static_cast<long>(s) * a.max_blocks + want + i - s_b[s]]);
  }
  for (int i = tid; i < need; i += ADV_THREADS) {
    const int s = adv_find(s_g, n, i);
    const int have = (s_old[s] + 127) >> 7;
    a.page_table[static_cast<long>(s) * a.max_blocks + have + i - s_g[s]] = checked(a.ring[wrap(head + i)]);
  }
  if (!maps) return;
  for (int r = tid; r < rows; r += ADV_THREADS) {
    const int s = adv_find(s_q, n, r);
    const int old = s_old[s], pos = old + r - s_q[s], b = pos >> 7, have = (old + 127) >> 7;
    const int page = checked(b < have ? a.page_table[static_cast<long>(s) * a.max_blocks + b]
                                      : a.ring[wrap(head + s_g[s] + b - have)]);
    a.slot_map[r] = page < 0 ? -1 : page * 128 + (pos & 127);
  }
}

// The slot map of a finished step; lanes take neighbouring rows, SLOT_ROWS of them a round with their loads in flight
// together.  A step that was refused has no rows.
__global__ void __launch_bounds__(SLOT_THREADS) slot_map_kernel(const AdvanceArgs a) {
  extern __shared__ int slot_smem[];                 // [num_seqs + 1] q_start
  const int n = a.num_seqs;
  pdl_wait();
  for (int s = threadIdx.x; s <= n; s += SLOT_THREADS) slot_smem[s] = a.q_start[s];
  __syncthreads();
  const int rows = slot_smem[n];
  for (int r0 = blockIdx.x * SLOT_THREADS * SLOT_ROWS + threadIdx.x; r0 < a.max_rows; r0 += gridDim.x * SLOT_THREADS * SLOT_ROWS) {
    int page[SLOT_ROWS], pos[SLOT_ROWS];
    int s = 0, next = -1;                            // next: first row behind sequence s
#pragma unroll
    for (int k = 0; k < SLOT_ROWS; ++k) {
      const int r = r0 + k * SLOT_THREADS;
      page[k] = -1;
      pos[k] = 0;
      if (r >= rows) continue;
      if (r >= next) {
        s = adv_find(slot_smem, n, r);
        next = slot_smem[s + 1];
      }
      pos[k] = a.ctx_out[s] - next + r;
      page[k] = a.page_table[static_cast<long>(s) * a.max_blocks + (pos[k] >> 7)];
    }
#pragma unroll
    for (int k = 0; k < SLOT_ROWS; ++k) {
      const int r = r0 + k * SLOT_THREADS;
      if (r >= a.max_rows) continue;
      const bool fine = page[k] >= 0 && page[k] < a.num_pages;
      if (!fine && r < rows) flag_error(MSA_DEV_BOUNDS);
      a.slot_map[r] = fine ? page[k] * 128 + (pos[k] & 127) : -1;
    }
  }
}

}  // namespace msa
