// Block-sparse decode attention (paged_sparse_attn): a cheap score chooses, for every sequence
// and KV head, the pages that the decode step reads.
//
// Score of page p for KV head g: the largest logit that its keys could give any of the group's
// queries, from the page's elementwise key bounds lo <= k <= hi:
//     s[b][g][p] = max_h sum_d max(q_hd lo_pd, q_hd hi_pd)
//                = max_h sum_d min(q_hd, 0) lo_pd + max(q_hd, 0) hi_pd,
// a product of the 2 d numbers (min(q, 0), max(q, 0)) with (lo, hi). Three steps:
//   score   warp-level mma.sync, 16 pages x 8 heads per tile; reads 4 d bytes per page and KV
//           head, 1/16 of the page's keys and values: HBM-bound.
//   select  one block per (sequence, KV head): the first `sink` and last `recent` pages, and the
//           best of the rest. The set is exactly that of the scores in 64 bits (ties to the
//           lower page): fp32 scores with a bound on their error decide all pages but those
//           near the border, and those are scored again in fp64.
//   attend  the streaming kernel over the chosen pages, and its join (stream.cu).
// 128 sequences of 2K to 16K slots, 28 query and 4 KV heads, 128 pages each: score 30 us (147 MB,
// 75 % of measured HBM), select 17 us, attend 95 to 98 us, join 7 us (from cold caches).
#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "paged_plan.cuh"
#include "row_items.cuh"

namespace kara {

namespace {

struct SparseArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* bounds;
  const int32_t* block_table;
  const int32_t* ctx_len;
  float2* score;        // [B, Hkv, max_blocks]: (score, sum of |terms|)
  int32_t* near_page;   // [B, Hkv, max_blocks]: pages near the border, ascending
  double* near_score;   // [B, Hkv, max_blocks]: their scores in fp64
  uint32_t* words;      // [B, Hkv, max_blocks / 32]: bitmaps too long for shared memory
  int32_t* sel;         // [B, Hkv, pages]
  int4* rows;           // [B]: the streaming kernel's line (cache row, 0, slots, start)
  int* total;
  int32_t* status;
  int B, Hq, Hkv, max_blocks, num_blocks, pages, sink, recent, extra;
};

// Length of sequence b in slots, and its pages.
__device__ __forceinline__ int seq_slots(const SparseArgs& a, int b) {
  const int64_t n = static_cast<int64_t>(a.ctx_len[b]) + a.extra;
  const int64_t top = static_cast<int64_t>(a.max_blocks) * 16;
  return static_cast<int>(n < 0 ? 0 : n > top ? top : n);
}
__device__ __forceinline__ int seq_pages(const SparseArgs& a, int b) {
  return (seq_slots(a, b) + 15) / 16;
}

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kScoreBlocks = 3;      // resident blocks per SM

// A warp takes tiles (sequence, 16 pages, KV head): A = the pages' bounds, read straight into
// fragments, B = the group's queries split by sign. The channel that a fragment slot stands for
// is free as long as A and B agree, so a lane takes 16 consecutive bytes of a row (8 channels,
// two k-steps) with each load. A second product of the absolute values gives sum |terms|, the
// scale of the score's error.
template <int D>
__global__ void __launch_bounds__(kScoreThreads, kScoreBlocks) page_score_kernel(const SparseArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int NC = D / 32;                     // 32-channel chunks of a bound row
  __shared__ RowItems<kScoreThreads> items;
  const int warp = warp_id(), lane = lane_id();
  const int grp = lane >> 2, tig = lane & 3;
  const int G = a.Hq / a.Hkv;
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kScoreWarps + warp;
  const int64_t num_warps = static_cast<int64_t>(gridDim.x) * kScoreWarps;
  if (blockIdx.x == 0) {                         // the line of selected pages, for the last step
    int start = 0;
    for (int b0 = 0; b0 < a.B; b0 += kScoreThreads) {
      const int bt = b0 + static_cast<int>(threadIdx.x);
      const int slots = bt < a.B ? seq_slots(a, bt) : 0;
      row_items_scan(items, min((slots + 15) / 16, a.pages));
      if (bt < a.B) a.rows[bt] = make_int4(bt, 0, slots, start + items.start[threadIdx.x]);
      start += items.start[kScoreThreads];
    }
    if (threadIdx.x == 0) *a.total = start;
  }
  int64_t base = 0;
  for (int b0 = 0; b0 < a.B; b0 += kScoreThreads) {
    const int bt = b0 + static_cast<int>(threadIdx.x);
    int count = 0;
    if (bt < a.B) {
      const int np = seq_pages(a, bt);
      // scores matter only where there is something to choose
      count = np > a.pages ? a.Hkv * ((np + 15) / 16) : 0;
    }
    row_items_scan(items, count);
    const int total = items.start[kScoreThreads];
    const int64_t skip =
        base <= gw ? gw - base : (num_warps - (base - gw) % num_warps) % num_warps;
    for (int64_t it = skip; it < total; it += num_warps) {
      const int row = row_items_find(items, static_cast<int>(it));
      const int b = b0 + row, local = static_cast<int>(it) - items.start[row];
      const int g = local % a.Hkv, p0 = local / a.Hkv * 16;
      const int np = seq_pages(a, b);
      // lanes 0..15 fetch the tile's block ids
      int blk = -1;
      if (lane < 16 && p0 + lane < np) {
        blk = a.block_table[static_cast<size_t>(b) * a.max_blocks + p0 + lane];
        if (blk < 0 || blk >= a.num_blocks) {
          report(a.status, KARA_ERR_BAD_BLOCK);
          blk = -1;
        }
      }
      const int blk_lo = __shfl_sync(0xffffffffu, blk, grp);
      const int blk_hi = __shfl_sync(0xffffffffu, blk, grp + 8);
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      const uint4* row_lo = reinterpret_cast<const uint4*>(
          a.bounds + (static_cast<size_t>(max(blk_lo, 0)) * a.Hkv + g) * 2 * D);
      const uint4* row_hi = reinterpret_cast<const uint4*>(
          a.bounds + (static_cast<size_t>(max(blk_hi, 0)) * a.Hkv + g) * 2 * D);
      uint4 x0[2 * NC], x1[2 * NC];
#pragma unroll
      for (int c = 0; c < 2 * NC; ++c) {
        x0[c] = blk_lo >= 0 ? row_lo[c * 4 + tig] : zero;
        x1[c] = blk_hi >= 0 ? row_hi[c * 4 + tig] : zero;
      }
      const uint4* qrow = reinterpret_cast<const uint4*>(
          a.q + (static_cast<size_t>(b) * a.Hq + g * G + (grp < G ? grp : 0)) * D);
      float s[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
      const __nv_bfloat162 none = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const uint4 qv = grp < G ? qrow[c * 4 + tig] : zero;
        const uint32_t qw[4] = {qv.x, qv.y, qv.z, qv.w};
        uint32_t neg[4], pos[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 t = *reinterpret_cast<const __nv_bfloat162*>(&qw[j]);
          const __nv_bfloat162 m = __hmin2(t, none), p = __hmax2(t, none);
          neg[j] = *reinterpret_cast<const uint32_t*>(&m);
          pos[j] = *reinterpret_cast<const uint32_t*>(&p);
        }
        const uint4 l0 = x0[c], l1 = x1[c], h0 = x0[NC + c], h1 = x1[NC + c];
        // four steps (64 terms) from zero: their errors stay those of 64 terms
        float t[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t k = 0x7fff7fffu;
        mma_bf16_16816(t, l0.x, l1.x, l0.y, l1.y, neg[0], neg[1]);
        mma_bf16_16816(e, l0.x & k, l1.x & k, l0.y & k, l1.y & k, neg[0] & k, neg[1] & k);
        mma_bf16_16816(t, l0.z, l1.z, l0.w, l1.w, neg[2], neg[3]);
        mma_bf16_16816(e, l0.z & k, l1.z & k, l0.w & k, l1.w & k, neg[2] & k, neg[3] & k);
        mma_bf16_16816(t, h0.x, h1.x, h0.y, h1.y, pos[0], pos[1]);
        mma_bf16_16816(e, h0.x & k, h1.x & k, h0.y & k, h1.y & k, pos[0] & k, pos[1] & k);
        mma_bf16_16816(t, h0.z, h1.z, h0.w, h1.w, pos[2], pos[3]);
        mma_bf16_16816(e, h0.z & k, h1.z & k, h0.w & k, h1.w & k, pos[2] & k, pos[3] & k);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += t[i];
      }
      // rows grp and grp + 8, heads 2 tig and 2 tig + 1: the maximum over the group's heads
      const bool h0 = 2 * tig < G, h1 = 2 * tig + 1 < G;
      float m0 = fmaxf(h0 ? s[0] : -INFINITY, h1 ? s[1] : -INFINITY);
      float m1 = fmaxf(h0 ? s[2] : -INFINITY, h1 ? s[3] : -INFINITY);
      float e0 = fmaxf(h0 ? e[0] : 0.f, h1 ? e[1] : 0.f);
      float e1 = fmaxf(h0 ? e[2] : 0.f, h1 ? e[3] : 0.f);
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, off));
        m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, off));
        e0 = fmaxf(e0, __shfl_xor_sync(0xffffffffu, e0, off));
        e1 = fmaxf(e1, __shfl_xor_sync(0xffffffffu, e1, off));
      }
      float2* dst = a.score + (static_cast<size_t>(b) * a.Hkv + g) * a.max_blocks + p0;
      // a page that the table does not hold goes last, as exact_score has it
      if (tig == 0 && p0 + grp < np) dst[grp] = make_float2(blk_lo >= 0 ? m0 : -INFINITY, e0);
      if (tig == 1 && p0 + grp + 8 < np)
        dst[grp + 8] = make_float2(blk_hi >= 0 ? m1 : -INFINITY, e1);
    }
    base += total;
  }
}

// Keys whose unsigned order is the order of the values; -0 as +0, NaN below everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_key(double x) {
  if (x != x) return 0ull;
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

constexpr int kListMinPages = 4;                 // selected pages that are worth a warp (128 of one
                                                 // sequence: 24.6 us, with 2 25.3, with 1 28.3)
constexpr int kSelBits = 10;
constexpr int kSelKeys = 4096;                   // pages whose keys stay in shared memory
constexpr int kDigit = 8;                        // bits of a score that one pass settles
constexpr int kDigitBins = 1 << kDigit;
constexpr int kSelFew = 64;                      // scores that are ranked by counting
constexpr int kSelBins = 1 << kSelBits;
constexpr int kSelList = 512;                    // candidates settled by counting
constexpr int kSelWords = 1024;                  // pages in the shared bitmap, / 32

template <int THREADS>
struct SelectSmem {
  int hist[kSelBins];
  unsigned long long list[kSelList];
  int list_page[kSelList];
  uint32_t words[kSelWords];
  uint32_t keys[kSelKeys];
  int warp_total[THREADS / 32];
  unsigned long long lo, hi;     // extreme keys
  uint32_t key_lo, key_hi;
  unsigned long long found;
  int bin, above, in_bin, total, count, sure, close;
  float err;
};

// Exclusive prefix sum over the block; s.total gets the sum.
template <int THREADS>
__device__ __forceinline__ int block_prefix(SelectSmem<THREADS>& s, int v) {
  const int lane = lane_id(), warp = warp_id();
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();
  if (lane == 31) s.warp_total[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int t = s.warp_total[w];
    before += w < warp ? t : 0;
    all += t;
  }
  if (threadIdx.x == 0) s.total = all;
  __syncthreads();
  return before + x - v;
}

// The k-th largest of the keys key(0 .. n-1), 1 <= k <= n, and how many keys exceed it. Radix
// selection from the highest bit in which the keys differ (scores of one row share sign and
// most exponent bits, so the first digit already spreads them over the bins); once a digit's bin
// holds few keys, those are ranked by counting. s.lo and s.hi hold the extreme keys.
template <int THREADS, typename KeyFn>
__device__ unsigned long long kth_largest(SelectSmem<THREADS>& s, int n, int k, const KeyFn& key,
                                          int& above) {
  const unsigned long long differ = s.lo ^ s.hi;
  int shift = differ == 0 ? 0 : 64 - __clzll(static_cast<long long>(differ));   // bits to settle
  unsigned long long prefix = shift < 64 ? s.hi >> shift : 0ull;                // settled bits
  above = 0;
  int rest = k;
  while (shift > 0) {
    const int bits = min(kSelBits, shift);
    const int next = shift - bits;
    __syncthreads();
    for (int i = threadIdx.x; i < kSelBins; i += THREADS) s.hist[i] = 0;
    if (threadIdx.x == 0) s.count = 0;
    __syncthreads();
#pragma unroll 8
    for (int i = threadIdx.x; i < n; i += THREADS) {
      const unsigned long long x = key(i);
      if ((shift < 64 ? x >> shift : 0ull) == prefix)
        atomicAdd(&s.hist[static_cast<int>(x >> next) & ((1 << bits) - 1)], 1);
    }
    __syncthreads();
    // bins from the top: thread t holds the kPer bins below those of the threads before it
    constexpr int kPer = kSelBins / THREADS;
    int mine[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      mine[j] = s.hist[kSelBins - 1 - (static_cast<int>(threadIdx.x) * kPer + j)];
      sum += mine[j];
    }
    int run = block_prefix(s, sum);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (run < rest && run + mine[j] >= rest) {
        s.bin = kSelBins - 1 - (static_cast<int>(threadIdx.x) * kPer + j);
        s.above = run;
        s.in_bin = mine[j];
      }
      run += mine[j];
    }
    __syncthreads();
    prefix = (prefix << bits) | static_cast<unsigned long long>(s.bin);
    above += s.above;
    rest -= s.above;
    shift = next;
    const int in_bin = s.in_bin;
    if (shift > 0 && in_bin <= min(kSelList, THREADS)) {
#pragma unroll 8
      for (int i = threadIdx.x; i < n; i += THREADS) {
        const unsigned long long x = key(i);
        if (x >> shift == prefix) s.list[atomicAdd(&s.count, 1)] = x;
      }
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < in_bin) {
        const unsigned long long x = s.list[threadIdx.x];
        int more = 0, same = 0;
        for (int j = 0; j < in_bin; ++j) {
          more += s.list[j] > x;
          same += s.list[j] == x;
        }
        if (more < rest && more + same >= rest) {   // equal keys write equal values
          s.found = x;
          s.above = more;
        }
      }
      __syncthreads();
      prefix = s.found;
      above += s.above;
      shift = 0;
    }
  }
  __syncthreads();
  return prefix;
}

// Extreme keys of this thread's keys into s.lo and s.hi (set to the empty range before).
template <int THREADS>
__device__ __forceinline__ void merge_extremes(SelectSmem<THREADS>& s, unsigned long long lo,
                                               unsigned long long hi) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const unsigned long long l2 = __shfl_xor_sync(0xffffffffu, lo, off);
    const unsigned long long h2 = __shfl_xor_sync(0xffffffffu, hi, off);
    lo = l2 < lo ? l2 : lo;
    hi = h2 > hi ? h2 : hi;
  }
  if (lane_id() == 0) {
    atomicMin(&s.lo, lo);
    atomicMax(&s.hi, hi);
  }
}
// Sets the empty range; ends with a barrier.
template <int THREADS>
__device__ __forceinline__ void clear_extremes(SelectSmem<THREADS>& s) {
  __syncthreads();
  if (threadIdx.x == 0) {
    s.lo = ~0ull;
    s.hi = 0ull;
  }
  __syncthreads();
}

// Error of an fp32 score, relative to the sum of its terms' magnitudes (e). It assumes that a
// tensor-core step adds 16 exact products to the sum so far and drops at most the bits below 2^-23
// of the largest of the 17 numbers, at most 17 * 2^-23 of it (how the hardware adds is not
// specified; the measured worst error, 2^-20 e, leaves a factor of 16). Over the four steps of a
// chain that is at most 68 * 2^-23 of the chain's e, over all chains 2^-16.9 e. The fp32 additions
// of the at most 4 chains are off by 2^-24 of partial sums below e each. e itself is summed in one
// chain, low by at most 2^-14 of its value.
constexpr float kScoreErr = 1.0f / 65536.0f;

// The largest of the group's exact scores of one page (a warp's work, every lane gets it). Four
// lanes per query head, each with every fourth 8-channel piece.
template <int D>
__device__ __forceinline__ double exact_score(const SparseArgs& a, int b, int g, int page) {
  const int G = a.Hq / a.Hkv;
  const int blk = a.block_table[static_cast<size_t>(b) * a.max_blocks + page];
  if (blk < 0 || blk >= a.num_blocks) return -INFINITY;
  const int h = lane_id() >> 2, part = lane_id() & 3;
  const uint4* lo = reinterpret_cast<const uint4*>(
      a.bounds + (static_cast<size_t>(blk) * a.Hkv + g) * 2 * D);
  const uint4* qr = reinterpret_cast<const uint4*>(
      a.q + (static_cast<size_t>(b) * a.Hq + g * G + min(h, G - 1)) * D);
  uint4 l[D / 32], u[D / 32], x[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    l[c] = lo[c * 4 + part];
    u[c] = lo[D / 8 + c * 4 + part];
    x[c] = qr[c * 4 + part];
  }
  double sum[2] = {0.0, 0.0};
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    const uint32_t* lw = reinterpret_cast<const uint32_t*>(&l[c]);
    const uint32_t* uw = reinterpret_cast<const uint32_t*>(&u[c]);
    const uint32_t* xw = reinterpret_cast<const uint32_t*>(&x[c]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      auto up = [](uint32_t w) { return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w)); };
      const float2 q = up(xw[j]), p = up(lw[j]), r = up(uw[j]);
      // a product of two bf16 numbers is exact in fp64
      sum[0] += static_cast<double>(q.x) * static_cast<double>(q.x < 0.f ? p.x : r.x);
      sum[1] += static_cast<double>(q.y) * static_cast<double>(q.y < 0.f ? p.y : r.y);
    }
  }
  double best = sum[0] + sum[1];
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) best += __shfl_xor_sync(0xffffffffu, best, off);
  if (h >= G || best != best) best = -INFINITY;
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    const double other = __shfl_xor_sync(0xffffffffu, best, off);
    best = other > best ? other : best;
  }
  return best;
}

// One block per (sequence, KV head). The chosen pages are a bitmap, so that they come out in
// ascending order from any order of work.
// What bounds it is latency: about 15 dependent steps (a load, a barrier, a first fetch of code
// each), 5 us for a row of 250 pages. 1024 threads where every block has an SM to itself and rows
// can be long (one sequence of 4K pages: its call 27.6 -> 25.3 us), else 512 (512 rows of 600 pages
// 149 us, with 1024 threads 158; 32 sequences of 257 pages 34.5 and 35.1; 256 threads gave 148 and
// 34.1, no more apart from 512 than two runs are). How long rows are only the device knows: the
// table's width bounds it, so a wide table takes 1024 threads for short rows too.
template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS) page_select_kernel(const SparseArgs a) {
  __shared__ SelectSmem<THREADS> s;
  const int bg = blockIdx.x, b = bg / a.Hkv, g = bg % a.Hkv;
  const int lane = lane_id();
  // What needs no scores comes before the wait for them: the lengths were written, and the last
  // call's lists read, before the score kernel was let start.
  auto follow = [] {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  };
  const int np = seq_pages(a, b);
  int32_t* sel = a.sel + static_cast<size_t>(bg) * a.pages;
  if (threadIdx.x == 0 && g == 0) {
    const int n_raw = a.ctx_len[b];
    if (n_raw < 0 || static_cast<int64_t>(n_raw) + a.extra > static_cast<int64_t>(a.max_blocks) * 16)
      report(a.status, KARA_ERR_INVALID_ARG);
  }
  if (np <= a.pages) {                           // everything fits
    for (int i = threadIdx.x; i < a.pages; i += THREADS) sel[i] = i < np ? i : -1;
    follow();
    return;
  }
  const int first = a.sink, last = np - a.recent;   // pages [first, last) compete
  const int want = a.pages - a.sink - a.recent;
  const int n = last - first;
  const float2* score = a.score + static_cast<size_t>(bg) * a.max_blocks + first;
  for (int i = threadIdx.x; i < a.sink; i += THREADS) sel[i] = i;
  for (int i = threadIdx.x; i < a.recent; i += THREADS) sel[a.sink + want + i] = last + i;
  if (want == 0) {
    follow();
    return;
  }
  int32_t* near_page = a.near_page + static_cast<size_t>(bg) * a.max_blocks;
  double* near_score = a.near_score + static_cast<size_t>(bg) * a.max_blocks;
  const int num_words = (n + 31) / 32;
  uint32_t* words = num_words <= kSelWords
                        ? s.words
                        : a.words + static_cast<size_t>(bg) * ((a.max_blocks + 31) / 32);

  // The row's scores as ordered keys, in shared memory where they fit. This kernel runs its code
  // once per block, so what it costs most is fetching it: little is unrolled.
  uint32_t* keys = n <= kSelKeys ? s.keys : reinterpret_cast<uint32_t*>(near_score);
  if (threadIdx.x == 0) {
    s.err = 0.f;
    s.sure = s.close = s.count = 0;
    s.key_lo = 0xffffffffu;
    s.key_hi = 0u;
  }
  // counts of a digit's values; a word of padding every 8 keeps a warp's scan free of conflicts
  auto slot = [](uint32_t bin) -> uint32_t { return bin + (bin >> 3); };
  constexpr int kSlots = kDigitBins + kDigitBins / 8;
#pragma unroll 1
  for (int i = threadIdx.x; i < kSlots; i += THREADS) s.hist[i] = 0;
  follow();
  float err = 0.f;
  uint32_t klo = 0xffffffffu, khi = 0u;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += THREADS) {
    const float2 x = score[i];
    const uint32_t k = order_key(x.x);
    keys[i] = k;
    klo = min(klo, k);
    khi = max(khi, k);
    err = x.y == x.y ? fmaxf(err, x.y) : INFINITY;
  }
  klo = __reduce_min_sync(0xffffffffu, klo);
  khi = __reduce_max_sync(0xffffffffu, khi);
  // magnitudes are not negative: they order as their bits
  const uint32_t eb = __reduce_max_sync(0xffffffffu, __float_as_uint(err));
  __syncthreads();
  if (lane == 0) {
    atomicMin(&s.key_lo, klo);
    atomicMax(&s.key_hi, khi);
    atomicMax(reinterpret_cast<unsigned int*>(&s.err), eb);
  }
  __syncthreads();

  // The want-th largest fp32 score: radix selection from the highest bit in which the scores
  // differ (they share sign and most exponent bits, so the first digit already spreads them),
  // until a bin holds few, which one warp ranks. The scans are a warp's too.
  uint32_t tkey;
  {
    const uint32_t differ = s.key_lo ^ s.key_hi;
    int shift = 32 - __clz(differ);              // bits to settle
    uint32_t prefix = shift < 32 ? s.key_hi >> shift : 0u;
    int rest = want;
    while (shift > 0) {
      const int bits = min(kDigit, shift), next = shift - bits;
#pragma unroll 4
      for (int i = threadIdx.x; i < n; i += THREADS) {
        const uint32_t k = keys[i];
        if ((shift < 32 ? k >> shift : 0u) == prefix)
          atomicAdd(&s.hist[slot((k >> next) & ((1u << bits) - 1))], 1);
      }
      __syncthreads();
      if (threadIdx.x < 32) {                    // values from the top, eight per lane
        int c[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          c[j] = s.hist[slot(kDigitBins - 1 - (lane * 8 + j))];
          sum += c[j];
        }
        int upto = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += y;
        }
        int run = upto - sum;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (run < rest && run + c[j] >= rest) {
            s.bin = kDigitBins - 1 - (lane * 8 + j);
            s.above = run;
            s.in_bin = c[j];
          }
          run += c[j];
        }
      }
      __syncthreads();
      prefix = (prefix << bits) | static_cast<uint32_t>(s.bin);
      rest -= s.above;
      shift = next;
      if (shift == 0) break;
      const int in_bin = s.in_bin;
      if (in_bin <= kSelFew) {
        uint32_t* list = reinterpret_cast<uint32_t*>(s.list);
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += THREADS)
          if (keys[i] >> shift == prefix) list[atomicAdd(&s.count, 1)] = keys[i];
        __syncthreads();
        for (int j0 = threadIdx.x; j0 < in_bin; j0 += THREADS) {
          const uint32_t mine = list[j0];
          int more = 0, same = 0;
          for (int j = 0; j < in_bin; ++j) {
            more += list[j] > mine;
            same += list[j] == mine;
          }
          if (more < rest && more + same >= rest) s.found = mine;   // equal keys: equal values
        }
        __syncthreads();
        prefix = static_cast<uint32_t>(s.found);
        shift = 0;
      } else {
        for (int i = threadIdx.x; i < kSlots; i += THREADS) s.hist[i] = 0;
        __syncthreads();
      }
    }
    tkey = prefix;
  }
  const float t = tkey == 0u ? __int_as_float(0x7fc00000)
                             : __uint_as_float((tkey & 0x80000000u) ? tkey ^ 0x80000000u : ~tkey);
  // the second part: fp32 products below 2^-126 may vanish, 2 d <= 256 of them
  const float margin = 2.f * kScoreErr * s.err + 1e-35f;
  // every page: surely among the best (a key above that of t + margin), surely not (below that of
  // t - margin), or near the border. An infinite margin says that fp32 sums overflowed, so that even
  // a score that is NaN in fp32 (the lowest key) may belong to the best: everything is near then, as
  // when t is NaN or infinite.
  const bool nan = !(margin < INFINITY) || !(t + margin == t + margin) || !(t - margin == t - margin);
  const uint32_t key_up = nan ? 0xffffffffu : order_key(t + margin);
  const uint32_t key_low = nan ? 0u : order_key(t - margin);
#pragma unroll 2
  for (int i0 = threadIdx.x - lane; i0 < num_words * 32; i0 += THREADS) {
    const int i = i0 + lane;
    const uint32_t k = i < n ? keys[i] : 0u;
    const bool sure = i < n && k > key_up;
    const bool close = i < n && !sure && k >= key_low;
    const uint32_t ws = __ballot_sync(0xffffffffu, sure), wc = __ballot_sync(0xffffffffu, close);
    if (lane == 0) {
      words[i0 / 32] = ws;
      if (ws != 0) atomicAdd(&s.sure, __popc(ws));
    }
    if (wc != 0) {
      int at = 0;
      if (lane == 0) at = atomicAdd(&s.close, __popc(wc));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(wc & ((1u << lane) - 1));
      if (close) {
        if (at < kSelList) s.list_page[at] = i;
        else near_page[at] = i;
      }
    }
  }
  __syncthreads();
  const int num_close = s.close, rest = want - s.sure;   // places left for the close pages
  // the close pages: the first kSelList in shared memory, the rest in the workspace
  auto close_page = [&](int j) -> int { return j < kSelList ? s.list_page[j] : near_page[j]; };
  if (rest >= num_close) {                       // all of them
    for (int j = threadIdx.x; j < num_close; j += THREADS) {
      const int i = close_page(j);
      atomicOr(&words[i / 32], 1u << (i & 31));
    }
  } else if (num_close <= min(kSelList, THREADS)) {
    for (int j = warp_id(); j < num_close; j += THREADS / 32) {
      const unsigned long long x = order_key(exact_score<D>(a, b, g, first + s.list_page[j]));
      if (lane == 0) s.list[j] = x;
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < num_close) {
      const int i = s.list_page[threadIdx.x];
      const unsigned long long x = s.list[threadIdx.x];
      int before = 0;                            // pages that go first
      for (int j = 0; j < num_close; ++j)
        before += s.list[j] > x || (s.list[j] == x && s.list_page[j] < i);
      if (before < rest) atomicOr(&words[i / 32], 1u << (i & 31));
    }
  } else {
    // many equal or nearly equal pages: select their exact scores the same way, then the lowest
    // pages among those equal to the last score that is taken
    clear_extremes(s);
    unsigned long long lo = ~0ull, hi = 0ull;
    for (int j = warp_id(); j < num_close; j += THREADS / 32) {
      const double e = exact_score<D>(a, b, g, first + close_page(j));
      if (lane == 0) near_score[j] = e;
      const unsigned long long x = order_key(e);
      lo = x < lo ? x : lo;
      hi = x > hi ? x : hi;
    }
    merge_extremes(s, lo, hi);
    __syncthreads();
    int over;
    const unsigned long long tc = kth_largest(
        s, num_close, rest, [&](int j) -> unsigned long long { return order_key(near_score[j]); },
        over);
    // pages equal to tc by falling page number; the others count as 0
    auto tie_key = [&](int j) -> unsigned long long {
      return order_key(near_score[j]) == tc ? 0xffffffffull - static_cast<uint32_t>(close_page(j))
                                            : 0ull;
    };
    clear_extremes(s);
    lo = ~0ull;
    hi = 0ull;
    for (int j = threadIdx.x; j < num_close; j += THREADS) {
      const unsigned long long x = tie_key(j);
      lo = x < lo ? x : lo;
      hi = x > hi ? x : hi;
    }
    merge_extremes(s, lo, hi);
    __syncthreads();
    int ignore;
    const unsigned long long edge = kth_largest(s, num_close, rest - over, tie_key, ignore);
    for (int j = threadIdx.x; j < num_close; j += THREADS) {
      if (order_key(near_score[j]) > tc || (tie_key(j) != 0 && tie_key(j) >= edge)) {
        const int i = close_page(j);
        atomicOr(&words[i / 32], 1u << (i & 31));
      }
    }
  }
  __syncthreads();
  // out in ascending order: one warp numbers the words' pages, every thread writes its own
  int* start = num_words <= kSelBins ? s.hist : near_page;   // the counts are no longer needed
  if (threadIdx.x < 32) {
    int carry = a.sink;
    for (int w0 = 0; w0 < num_words; w0 += 32) {
      const int w = w0 + lane;
      const int mine = w < num_words ? __popc(words[w]) : 0;
      int upto = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += y;
      }
      if (w < num_words) start[w] = carry + upto - mine;
      carry += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  __syncthreads();
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += THREADS) {
    const uint32_t bits = words[i / 32], bit = 1u << (i & 31);
    if (bits & bit) sel[start[i / 32] + __popc(bits & (bit - 1))] = first + i;
  }
}

size_t align_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct SparseLayout {
  size_t head, rows, part_o, part_ml, score, near_score, near_page, words, sel, total;
};
SparseLayout sparse_layout(int B, int Hq, int Hkv, int D, int max_blocks, int pages) {
  SparseLayout l;
  const size_t rows = static_cast<size_t>(B) * Hkv;
  const size_t parts = (static_cast<size_t>(B) + stream_max_ranges(Hkv)) * Hq;
  l.head = 0;
  l.rows = 256;
  l.part_o = align_up(l.rows + static_cast<size_t>(B) * sizeof(int4));
  l.part_ml = align_up(l.part_o + parts * D * sizeof(float));
  l.score = align_up(l.part_ml + parts * sizeof(float2));
  l.near_score = align_up(l.score + rows * max_blocks * sizeof(float2));
  l.near_page = align_up(l.near_score + rows * max_blocks * sizeof(double));
  l.words = align_up(l.near_page + rows * max_blocks * sizeof(int32_t));
  l.sel = align_up(l.words + rows * ((max_blocks + 31) / 32) * sizeof(uint32_t));
  l.total = align_up(l.sel + rows * pages * sizeof(int32_t));
  return l;
}

template <int D>
kara_status launch_sparse_d(const SparseArgs& a, cudaStream_t stream) {
  int sms = 148;
  const int dev = device_slot();
  if (dev >= 0) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // no sequence has pages to choose from when all of them fit: one block writes the line
  const int64_t tiles = a.max_blocks > a.pages
                            ? static_cast<int64_t>(a.B) * a.Hkv * ((a.max_blocks + 15) / 16)
                            : 1;
  const int64_t most = (tiles + kScoreWarps - 1) / kScoreWarps;
  const int64_t wave = static_cast<int64_t>(sms) * kScoreBlocks;
  launch_pdl(page_score_kernel<D>, dim3(static_cast<unsigned>(most < wave ? most : wave)),
             dim3(kScoreThreads), 0, stream, a);
  const dim3 rows(static_cast<unsigned>(a.B * a.Hkv));
  if (static_cast<int64_t>(a.B) * a.Hkv <= sms && a.max_blocks > 1024)
    launch_pdl(page_select_kernel<D, 1024>, rows, dim3(1024), 0, stream, a);
  else
    launch_pdl(page_select_kernel<D, 512>, rows, dim3(512), 0, stream, a);
  return check_launch("paged_sparse_attn");
}

}  // namespace

size_t sparse_workspace_bytes(int B, int Hq, int Hkv, int D, int max_blocks, int pages) {
  return sparse_layout(B, Hq, Hkv, D, max_blocks, std::min(pages, max_blocks)).total;
}

kara_status launch_sparse(const SparseLaunch& L, cudaStream_t stream) {
  const SparseLayout lay = sparse_layout(L.B, L.Hq, L.Hkv, L.D, L.max_blocks,
                                         std::min(L.pages, L.max_blocks));
  // the caller's lists have num_pages entries each, the workspace's no more than the table (where
  // every page is read, as every page then fits)
  const int pages = L.sel != nullptr ? L.pages : std::min(L.pages, L.max_blocks);
  uint8_t* ws = static_cast<uint8_t*>(L.workspace);
  SparseArgs a;
  a.q = static_cast<const __nv_bfloat16*>(L.q);
  a.bounds = static_cast<const __nv_bfloat16*>(L.bounds);
  a.block_table = L.block_table;
  a.ctx_len = L.ctx_len;
  a.score = reinterpret_cast<float2*>(ws + lay.score);
  a.near_page = reinterpret_cast<int32_t*>(ws + lay.near_page);
  a.near_score = reinterpret_cast<double*>(ws + lay.near_score);
  a.words = reinterpret_cast<uint32_t*>(ws + lay.words);
  a.sel = L.sel != nullptr ? L.sel : reinterpret_cast<int32_t*>(ws + lay.sel);
  a.rows = reinterpret_cast<int4*>(ws + lay.rows);
  a.total = reinterpret_cast<int*>(ws + lay.head);
  a.status = L.status;
  a.B = L.B;
  a.Hq = L.Hq;
  a.Hkv = L.Hkv;
  a.max_blocks = L.max_blocks;
  a.num_blocks = L.num_blocks;
  a.pages = pages;
  a.sink = L.sink;
  a.recent = L.recent;
  a.extra = L.new_slots;
  kara_status st = L.D == 128 ? launch_sparse_d<128>(a, stream) : launch_sparse_d<64>(a, stream);
  if (st != KARA_OK) return st;
  StreamLaunch t;
  t.q = L.q;
  t.k_cache = L.k_cache;
  t.v_cache = L.v_cache;
  t.block_table = L.block_table;
  t.status = L.status;
  t.sel = a.sel;
  t.sel_pages = pages;
  t.line.rows = a.rows;
  t.line.total = a.total;
  t.line.max_ranges = 0;
  t.line.min_pages = kListMinPages;
  t.part_o = reinterpret_cast<float*>(ws + lay.part_o);
  t.part_ml = reinterpret_cast<float2*>(ws + lay.part_ml);
  t.B = L.B;
  t.Hq = L.Hq;
  t.Hkv = L.Hkv;
  t.D = L.D;
  t.max_blocks = L.max_blocks;
  t.num_blocks = L.num_blocks;
  t.scale = L.scale;
  t.beside = false;
  if ((st = launch_stream(&t, stream)) != KARA_OK) return st;
  JoinLaunch j = {};
  j.line = t.line;
  j.part_o = t.part_o;
  j.part_ml = t.part_ml;
  j.out = L.out;
  j.B = L.B;
  j.Hq = L.Hq;
  j.Hkv = L.Hkv;
  j.D = L.D;
  return launch_join(j, stream);
}

}  // namespace kara
