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
//   attend  the streaming decode kernel over the chosen pages, and its combine.
#include <cstdint>

#include "common.cuh"
#include "internal.h"
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
  int32_t* sel;         // [B, Hkv, pages]
  int32_t* status;
  int B, Hq, Hkv, max_blocks, num_blocks, pages, sink, recent, extra;
};

// Length of sequence b in slots, and its pages.
__device__ __forceinline__ int seq_pages(const SparseArgs& a, int b) {
  const int64_t n = static_cast<int64_t>(a.ctx_len[b]) + a.extra;
  const int64_t top = static_cast<int64_t>(a.max_blocks) * 16;
  return static_cast<int>(((n < 0 ? 0 : n > top ? top : n) + 15) / 16);
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

// A warp takes tiles (sequence, 16 pages, KV head): A = the pages' bounds, read straight into
// fragments, B = the group's queries split by sign. The channel that a fragment slot stands for
// is free as long as A and B agree, so a lane takes 16 consecutive bytes of a row (8 channels,
// two k-steps) with each load. A second product of the absolute values gives sum |terms|, the
// scale of the score's error.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const SparseArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int NC = D / 32;                     // 32-channel chunks of a bound row
  __shared__ RowItems<kScoreThreads> items;
  const int warp = warp_id(), lane = lane_id();
  const int grp = lane >> 2, tig = lane & 3;
  const int G = a.Hq / a.Hkv;
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kScoreWarps + warp;
  const int64_t num_warps = static_cast<int64_t>(gridDim.x) * kScoreWarps;
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
        uint32_t neg[4], pos[4], mag[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 t = *reinterpret_cast<const __nv_bfloat162*>(&qw[j]);
          const __nv_bfloat162 m = __hmin2(t, none), p = __hmax2(t, none);
          neg[j] = *reinterpret_cast<const uint32_t*>(&m);
          pos[j] = *reinterpret_cast<const uint32_t*>(&p);
          mag[j] = qw[j] & 0x7fff7fffu;
        }
        const uint4 l0 = x0[c], l1 = x1[c], h0 = x0[NC + c], h1 = x1[NC + c];
        mma_bf16_16816(s, l0.x, l1.x, l0.y, l1.y, neg[0], neg[1]);
        mma_bf16_16816(s, l0.z, l1.z, l0.w, l1.w, neg[2], neg[3]);
        mma_bf16_16816(s, h0.x, h1.x, h0.y, h1.y, pos[0], pos[1]);
        mma_bf16_16816(s, h0.z, h1.z, h0.w, h1.w, pos[2], pos[3]);
        // |q| (|lo| + |hi|) >= the terms' magnitudes
        const uint32_t k = 0x7fff7fffu;
        mma_bf16_16816(e, l0.x & k, l1.x & k, l0.y & k, l1.y & k, mag[0], mag[1]);
        mma_bf16_16816(e, l0.z & k, l1.z & k, l0.w & k, l1.w & k, mag[2], mag[3]);
        mma_bf16_16816(e, h0.x & k, h1.x & k, h0.y & k, h1.y & k, mag[0], mag[1]);
        mma_bf16_16816(e, h0.z & k, h1.z & k, h0.w & k, h1.w & k, mag[2], mag[3]);
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
      if (tig == 0 && p0 + grp < np) dst[grp] = make_float2(m0, e0);
      if (tig == 1 && p0 + grp + 8 < np) dst[grp + 8] = make_float2(m1, e1);
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

constexpr int kSelThreads = 512;
constexpr int kSelBits = 11;
constexpr int kSelBins = 1 << kSelBits;

struct SelectSmem {
  int hist[kSelBins];
  int warp_total[kSelThreads / 32];
  unsigned long long lo, hi;     // extreme keys
  int bin, above, total;
  float err;
};

// Exclusive prefix sum over the block; s.total gets the sum.
__device__ __forceinline__ int block_prefix(SelectSmem& s, int v) {
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
  for (int w = 0; w < kSelThreads / 32; ++w) {
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
// most exponent bits, so the first digit already spreads them over the bins).
template <typename Key, typename KeyFn>
__device__ Key kth_largest(SelectSmem& s, int n, int k, const KeyFn& key, int& above) {
  __syncthreads();
  if (threadIdx.x == 0) {
    s.lo = ~0ull;
    s.hi = 0ull;
  }
  __syncthreads();
  unsigned long long lo = ~0ull, hi = 0ull;
  for (int i = threadIdx.x; i < n; i += kSelThreads) {
    const unsigned long long x = key(i);
    lo = x < lo ? x : lo;
    hi = x > hi ? x : hi;
  }
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
  __syncthreads();
  const unsigned long long differ = s.lo ^ s.hi;
  int shift = differ == 0 ? 0 : 64 - __clzll(static_cast<long long>(differ));   // bits to settle
  unsigned long long prefix = shift < 64 ? s.hi >> shift : 0ull;                // settled bits
  above = 0;
  int rest = k;
  while (shift > 0) {
    const int bits = min(kSelBits, shift);
    const int next = shift - bits;
    __syncthreads();
    for (int i = threadIdx.x; i < kSelBins; i += kSelThreads) s.hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kSelThreads) {
      const unsigned long long x = key(i);
      if ((shift < 64 ? x >> shift : 0ull) == prefix)
        atomicAdd(&s.hist[static_cast<int>(x >> next) & ((1 << bits) - 1)], 1);
    }
    __syncthreads();
    // bins from the top: thread t holds bins [B - 4(t+1), B - 4t)
    constexpr int kPer = kSelBins / kSelThreads;
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
      }
      run += mine[j];
    }
    __syncthreads();
    prefix = (prefix << bits) | static_cast<unsigned long long>(s.bin);
    above += s.above;
    rest -= s.above;
    shift = next;
  }
  __syncthreads();
  return static_cast<Key>(prefix);
}

// Error of an fp32 score, relative to the sum of its terms' magnitudes: 2 d <= 256 terms enter
// 16 tensor-core steps; each step adds 17 numbers whose alignment may drop bits below 2^-23 of
// the largest, at most 16 * 17 * 2^-23 = 2^-14.9 in all, and the magnitudes themselves are
// computed as (|lo| + |hi|) |q| >= them with the same relative error.
constexpr float kScoreErr = 1.0f / 16384.0f;

// One block per (sequence, KV head). Thread t looks at a run of consecutive pages, so that one
// prefix sum over the threads orders the output.
template <int D>
__global__ void __launch_bounds__(kSelThreads) page_select_kernel(const SparseArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ SelectSmem s;
  const int bg = blockIdx.x, b = bg / a.Hkv, g = bg % a.Hkv;
  const int np = seq_pages(a, b);
  int32_t* sel = a.sel + static_cast<size_t>(bg) * a.pages;
  if (threadIdx.x == 0 && g == 0) {
    const int n_raw = a.ctx_len[b];
    if (n_raw < 0 || static_cast<int64_t>(n_raw) + a.extra > static_cast<int64_t>(a.max_blocks) * 16)
      report(a.status, KARA_ERR_INVALID_ARG);
  }
  if (np <= a.pages) {                           // everything fits
    for (int i = threadIdx.x; i < a.pages; i += kSelThreads) sel[i] = i < np ? i : -1;
    return;
  }
  const int first = a.sink, last = np - a.recent;   // pages [first, last) compete
  const int want = a.pages - a.sink - a.recent;
  const int n = last - first;
  const float2* score = a.score + static_cast<size_t>(bg) * a.max_blocks + first;
  int32_t* near_page = a.near_page + static_cast<size_t>(bg) * a.max_blocks;
  double* near_score = a.near_score + static_cast<size_t>(bg) * a.max_blocks;
  for (int i = threadIdx.x; i < a.sink; i += kSelThreads) sel[i] = i;
  for (int i = threadIdx.x; i < a.recent; i += kSelThreads) sel[a.sink + want + i] = last + i;
  if (want == 0) return;

  // the want-th largest fp32 score, and the error that any score of the row may have
  int above;
  const uint32_t tkey = kth_largest<uint32_t>(
      s, n, want, [&](int i) -> unsigned long long { return order_key(score[i].x); }, above);
  const float t = tkey == 0u ? __int_as_float(0x7fc00000)
                             : __uint_as_float((tkey & 0x80000000u) ? tkey ^ 0x80000000u : ~tkey);
  float err = 0.f;
  if (threadIdx.x == 0) s.err = 0.f;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kSelThreads) {
    const float e = score[i].y;
    err = e == e ? fmaxf(err, e) : INFINITY;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    err = fmaxf(err, __shfl_xor_sync(0xffffffffu, err, off));
  if (lane_id() == 0) atomicMax(reinterpret_cast<int*>(&s.err), __float_as_int(err));
  __syncthreads();
  const float margin = 2.f * kScoreErr * s.err;
  // > 0: certainly among the best; < 0: certainly not; 0: near the border
  auto side = [&](int i) -> int {
    const float x = score[i].x;
    return x > t + margin ? 1 : x < t - margin ? -1 : 0;
  };
  const int per = (n + kSelThreads - 1) / kSelThreads;
  const int i0 = min(n, static_cast<int>(threadIdx.x) * per), i1 = min(n, i0 + per);
  int sure = 0, close = 0;
  for (int i = i0; i < i1; ++i) {
    const int c = side(i);
    sure += c > 0;
    close += c == 0;
  }
  block_prefix(s, sure);
  const int rest = want - s.total;               // places left for the close ones
  const int close0 = block_prefix(s, close);
  const int num_close = s.total;
  // close pages in ascending order; scored in fp64 unless all of them are wanted
  uint64_t tc = 0;
  int ties = num_close;                          // how many equal to tc are taken
  const bool judge = rest < num_close;
  if (judge) {
    int at = close0;
    for (int i = i0; i < i1; ++i)
      if (side(i) == 0) near_page[at++] = first + i;
    __syncthreads();
    const int G = a.Hq / a.Hkv;
    for (int j = warp_id(); j < num_close; j += kSelThreads / 32) {
      const int page = near_page[j];
      const int blk = a.block_table[static_cast<size_t>(b) * a.max_blocks + page];
      double best = -INFINITY;
      if (blk >= 0 && blk < a.num_blocks) {
        const __nv_bfloat16* lo = a.bounds + (static_cast<size_t>(blk) * a.Hkv + g) * 2 * D;
        for (int h = 0; h < G; ++h) {
          const __nv_bfloat16* q = a.q + (static_cast<size_t>(b) * a.Hq + g * G + h) * D;
          double sum = 0.0;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const int d = c * 32 + lane_id();
            const float x = __bfloat162float(q[d]);
            const float y = __bfloat162float(x < 0.f ? lo[d] : lo[D + d]);
            // a product of two bf16 numbers is exact in fp64
            sum += static_cast<double>(x) * static_cast<double>(y);
          }
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          best = sum > best ? sum : best;
        }
      }
      if (lane_id() == 0) near_score[j] = best;
    }
    __syncthreads();
    int over;
    tc = kth_largest<uint64_t>(
        s, num_close, rest, [&](int i) -> unsigned long long { return order_key(near_score[i]); },
        over);
    ties = rest - over;
  }
  // among the close pages equal to tc the first `ties` are taken
  int equal = 0;
  if (judge)
    for (int j = close0; j < close0 + close; ++j) equal += order_key(near_score[j]) == tc;
  else
    equal = close;
  const int equal0 = block_prefix(s, equal);
  int emit = sure + max(0, min(equal, ties - equal0));
  if (judge)
    for (int j = close0; j < close0 + close; ++j) emit += order_key(near_score[j]) > tc;
  int out = a.sink + block_prefix(s, emit);
  int j = close0, eq = equal0;
  for (int i = i0; i < i1; ++i) {
    const int c = side(i);
    bool take = c > 0;
    if (c == 0) {
      if (judge) {
        const uint64_t x = order_key(near_score[j]);
        take = x > tc || (x == tc && eq++ < ties);
      } else {
        take = eq++ < ties;
      }
      ++j;
    }
    if (take) sel[out++] = first + i;
  }
}

size_t align_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct SparseLayout {
  size_t decode, score, near_score, near_page, sel, total;
};
SparseLayout sparse_layout(int B, int Hq, int Hkv, int D, int max_blocks, int pages) {
  SparseLayout l;
  const size_t rows = static_cast<size_t>(B) * Hkv;
  l.decode = 0;
  l.score = align_up(decode_workspace_bytes(B, Hq, D, pages));
  l.near_score = align_up(l.score + rows * max_blocks * sizeof(float2));
  l.near_page = align_up(l.near_score + rows * max_blocks * sizeof(double));
  l.sel = align_up(l.near_page + rows * max_blocks * sizeof(int32_t));
  l.total = align_up(l.sel + rows * pages * sizeof(int32_t));
  return l;
}

template <int D>
kara_status launch_sparse_d(const SparseArgs& a, cudaStream_t stream) {
  if (a.max_blocks > a.pages) {                  // some sequence may have pages to choose from
    int sms = 148;
    const int dev = device_slot();
    if (dev >= 0) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t tiles = static_cast<int64_t>(a.B) * a.Hkv * ((a.max_blocks + 15) / 16);
    const int64_t most = (tiles + kScoreWarps - 1) / kScoreWarps;
    const int64_t wave = static_cast<int64_t>(sms) * 2;
    launch_pdl(page_score_kernel<D>, dim3(static_cast<unsigned>(most < wave ? most : wave)),
               dim3(kScoreThreads), 0, stream, a);
  }
  launch_pdl(page_select_kernel<D>, dim3(static_cast<unsigned>(a.B * a.Hkv)), dim3(kSelThreads),
             0, stream, a);
  return check_launch("paged_sparse_attn");
}

}  // namespace

size_t sparse_workspace_bytes(int B, int Hq, int Hkv, int D, int max_blocks, int pages) {
  return sparse_layout(B, Hq, Hkv, D, max_blocks, pages).total;
}

kara_status launch_sparse(const SparseLaunch& L, cudaStream_t stream) {
  const SparseLayout lay = sparse_layout(L.B, L.Hq, L.Hkv, L.D, L.max_blocks, L.pages);
  uint8_t* ws = static_cast<uint8_t*>(L.workspace);
  SparseArgs a;
  a.q = static_cast<const __nv_bfloat16*>(L.q);
  a.bounds = static_cast<const __nv_bfloat16*>(L.bounds);
  a.block_table = L.block_table;
  a.ctx_len = L.ctx_len;
  a.score = reinterpret_cast<float2*>(ws + lay.score);
  a.near_page = reinterpret_cast<int32_t*>(ws + lay.near_page);
  a.near_score = reinterpret_cast<double*>(ws + lay.near_score);
  a.sel = L.sel != nullptr ? L.sel : reinterpret_cast<int32_t*>(ws + lay.sel);
  a.status = L.status;
  a.B = L.B;
  a.Hq = L.Hq;
  a.Hkv = L.Hkv;
  a.max_blocks = L.max_blocks;
  a.num_blocks = L.num_blocks;
  a.pages = L.pages;
  a.sink = L.sink;
  a.recent = L.recent;
  a.extra = L.new_slots;
  const kara_status st = L.D == 128 ? launch_sparse_d<128>(a, stream) : launch_sparse_d<64>(a, stream);
  if (st != KARA_OK) return st;
  DecodeLaunch d;
  d.q = L.q;
  d.k_cache = L.k_cache;
  d.v_cache = L.v_cache;
  d.block_table = L.block_table;
  d.ctx_len = L.ctx_len;
  d.out = L.out;
  d.partial = reinterpret_cast<float*>(ws + lay.decode);
  d.status = L.status;
  d.B = L.B;
  d.Hq = L.Hq;
  d.Hkv = L.Hkv;
  d.D = L.D;
  d.max_blocks = L.max_blocks;
  d.num_blocks = L.num_blocks;
  d.scale = L.scale;
  d.extra = L.new_slots;
  d.sel = a.sel;
  d.sel_pages = L.pages;
  return launch_decode(d, stream);
}

}  // namespace kara
