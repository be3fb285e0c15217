// New tokens entering the paged cache: rotary position embedding of their queries and keys on
// the way (paged_rope_append), and the per-page key bounds that block-sparse attention scores
// (paged_page_bounds).
//
// Rotation of a pair (x, y) of channels by the angle a = position * inv_freq[pair]:
//     x' = x cos a - y sin a,   y' = y cos a + x sin a,
// in fp32, rounded once to bf16. The angle is taken in turns, a / 2 pi = position *
// (inv_freq / 2 pi) in fp64, and reduced to [-1/2, 1/2] there before the fp32 sine and cosine:
// fp32 products lose the angle of far positions (at position 10^6 by 0.06 radians), fp64 turns
// keep it to 5e-7 radians over all int32 positions. Positions are an input of their own: after
// a compression a slot's number is no longer its token's position.
//
// Both kernels move every byte once: HBM-bound for prompts and caches, launch latency for a
// decode step. Measured: 12.7K prompt tokens of 28 + 2 * 4 heads 48.6 us, 4.85 TB/s (74 % of
// measured; the sines cost 4 us, the bounds 1 us), one token 3.7 us, 128 tokens 4.4 us; bounds of
// 636K slots 118 us, 6.2 TB/s (94 %).
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "row_items.cuh"

namespace kara {

namespace {

constexpr int kAppThreads = 256;
// Heads a thread has in flight: 192 bytes of loads (4 heads were 6 % slower on prompts; three
// blocks per SM with 2 or 3 heads 1 to 6 %; blocks that share an item's heads 30 %, for they
// repeat its sines and look-ups).
constexpr int kAppBatch = 6;

struct AppendArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t q_stride, k_stride, v_stride;   // elements between tokens
  const int32_t* cu;                      // [B + 1] or null (one token per sequence)
  const int32_t* positions;
  const float* inv_freq;
  __nv_bfloat16* k_cache;
  __nv_bfloat16* v_cache;
  __nv_bfloat16* bounds;                  // [num_blocks, Hkv, 2, D] or null
  __nv_bfloat16* q_ring;                  // [B, 2W, Hq, D] or null
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;                   // [T, Hkv, D] or null
  const int32_t* block_table;
  const int32_t* ctx_len;
  int32_t* status;
  int T, B, Hq, Hkv, max_blocks, num_blocks, rd, ring_w;
};

// Smallest and largest of the 16 rows of a page, 8 channels of one KV head. The page may have
// been written by this block just before, so the loads are ordinary ones.
__device__ __forceinline__ void page_bounds_unit(const __nv_bfloat16* k_cache,
                                                 __nv_bfloat16* bounds, int blk, int Hkv, int D,
                                                 int unit) {
  const int per_head = D / 8;
  const int g = unit / per_head, c = unit % per_head;
  const size_t row = static_cast<size_t>(Hkv) * D;
  const __nv_bfloat16* src = k_cache + static_cast<size_t>(blk) * 16 * row +
                             static_cast<size_t>(g) * D + c * 8;
  uint4 x[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) x[r] = *reinterpret_cast<const uint4*>(src + r * row);
  uint4 lo = x[0], hi = x[0];
  auto fold = [](uint32_t& a, uint32_t b, bool mx) {
    const __nv_bfloat162 va = *reinterpret_cast<__nv_bfloat162*>(&a);
    const __nv_bfloat162 vb = *reinterpret_cast<__nv_bfloat162*>(&b);
    const __nv_bfloat162 r = mx ? __hmax2(va, vb) : __hmin2(va, vb);
    a = *reinterpret_cast<const uint32_t*>(&r);
  };
#pragma unroll
  for (int r = 1; r < 16; ++r) {
    fold(lo.x, x[r].x, false);
    fold(lo.y, x[r].y, false);
    fold(lo.z, x[r].z, false);
    fold(lo.w, x[r].w, false);
    fold(hi.x, x[r].x, true);
    fold(hi.y, x[r].y, true);
    fold(hi.z, x[r].z, true);
    fold(hi.w, x[r].w, true);
  }
  __nv_bfloat16* dst = bounds + (static_cast<size_t>(blk) * Hkv + g) * 2 * D + c * 8;
  *reinterpret_cast<uint4*>(dst) = lo;
  *reinterpret_cast<uint4*>(dst + D) = hi;
}

// One work item = the new tokens of one sequence that fall into one page (at most 16), so that
// a page this call completes is complete within one block and its bounds can follow at once.
// A thread owns 16 channels of one token (two 16-byte vectors that hold 8 rotation pairs),
// whose sines it needs for every head, and walks the heads: queries, keys, then values.
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppThreads, 2) rope_append_kernel(const AppendArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int U = D / 16;                      // 16-channel units per head
  constexpr int kGroups = kAppThreads / U;
  __shared__ RowItems<kAppThreads> items;
  __shared__ float s_cos[16][D / 2], s_sin[16][D / 2];
  const int half = a.rd / 2;
  const int u = threadIdx.x % U, grp = threadIdx.x / U;
  const bool turns = u < a.rd / 16;              // this unit holds rotated channels
  int oa, ob;                                    // the unit's two 8-channel vectors
  if (INTERLEAVED || !turns) {
    oa = INTERLEAVED ? 16 * u : a.rd + 16 * (u - a.rd / 16);
    ob = oa + 8;
  } else {
    oa = 8 * u;
    ob = half + 8 * u;
  }

  // tokens n0 .. n0 + nb of sequence b, their first packed row t0
  auto tokens = [&](int b, int& t0) -> int {
    if (a.cu == nullptr) {
      t0 = b;
      return 1;
    }
    const int lo = a.cu[b], hi = a.cu[b + 1];
    t0 = lo;
    if (lo < 0 || hi < lo || hi > a.T) {
      report(a.status, KARA_ERR_INVALID_ARG);
      return 0;
    }
    return hi - lo;
  };
  const int table_slots = a.max_blocks * 16;

  int64_t base = 0;
  for (int b0 = 0; b0 < a.B; b0 += kAppThreads) {
    const int bt = b0 + static_cast<int>(threadIdx.x);
    int count = 0;
    if (bt < a.B) {
      int t0;
      const int nb = tokens(bt, t0);
      const int off = min(max(a.ctx_len[bt], 0), table_slots) % 16;
      count = nb > 0 ? (off + nb - 1) / 16 + 1 : 0;
    }
    row_items_scan(items, count);
    const int total = items.start[kAppThreads];
    // this block's items of the chunk: global numbers blockIdx.x, + gridDim.x, ...
    const int64_t skip = base <= static_cast<int64_t>(blockIdx.x)
                             ? static_cast<int64_t>(blockIdx.x) - base
                             : (gridDim.x - (base - blockIdx.x) % gridDim.x) % gridDim.x;
    for (int64_t it = skip; it < total; it += gridDim.x) {
      const int row = row_items_find(items, static_cast<int>(it));
      const int b = b0 + row, run = static_cast<int>(it) - items.start[row];
      int t_first;
      const int nb = tokens(b, t_first);
      const int n_raw = a.ctx_len[b];
      const int n0 = min(max(n_raw, 0), table_slots);
      const int page = n0 / 16 + run;
      const int s_lo = max(n0, page * 16), s_hi = min(n0 + nb, page * 16 + 16);
      const int c = s_hi - s_lo;
      const int t0 = t_first + s_lo - n0;
      int blk = -1;
      const bool in_table = n_raw == n0 && page < a.max_blocks;
      if (in_table) {
        blk = a.block_table[static_cast<size_t>(b) * a.max_blocks + page];
        if (blk < 0 || blk >= a.num_blocks) {
          if (threadIdx.x == 0) report(a.status, KARA_ERR_BAD_BLOCK);
          blk = -1;
        }
      } else if (threadIdx.x == 0) {
        report(a.status, KARA_ERR_INVALID_ARG);
      }
      __syncthreads();                           // the previous item's sines are no longer read
      for (int i = threadIdx.x; i < c * half; i += kAppThreads) {
        const int tok = i / half, f = i - tok * half;
        const double turn = static_cast<double>(a.positions[t0 + tok]) *
                            (static_cast<double>(a.inv_freq[f]) * 0.15915494309189535);
        const float x = static_cast<float>(turn - rint(turn));
        sincospif(2.f * x, &s_sin[tok][f], &s_cos[tok][f]);
      }
      __syncthreads();
      const int nsub = kGroups / c;
      const int tok = grp % c, sub = grp / c;
      if (sub < nsub) {
        const int t = t0 + tok, slot = s_lo + tok;
        float cs[8], sn[8];
        if (turns) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            cs[j] = s_cos[tok][8 * u + j];
            sn[j] = s_sin[tok][8 * u + j];
          }
        }
        const size_t cache_row = (static_cast<size_t>(blk < 0 ? 0 : blk) * 16 + slot % 16) *
                                 a.Hkv * D;
        // of several tokens that share a ring row the last one stays
        const bool ring = a.q_ring != nullptr && in_table && slot >= n0 + nb - a.ring_w;
        const int heads = a.Hq + 2 * a.Hkv;
        for (int h0 = sub; h0 < heads; h0 += nsub * kAppBatch) {
          uint4 xa[kAppBatch], xb[kAppBatch];
#pragma unroll
          for (int i = 0; i < kAppBatch; ++i) {
            const int h = h0 + i * nsub;
            if (h < heads) {
              const __nv_bfloat16* src =
                  h < a.Hq ? a.q + t * a.q_stride + static_cast<int64_t>(h) * D
                  : h < a.Hq + a.Hkv
                      ? a.k + t * a.k_stride + static_cast<int64_t>(h - a.Hq) * D
                      : a.v + t * a.v_stride + static_cast<int64_t>(h - a.Hq - a.Hkv) * D;
              xa[i] = *reinterpret_cast<const uint4*>(src + oa);
              xb[i] = *reinterpret_cast<const uint4*>(src + ob);
            }
          }
#pragma unroll
          for (int i = 0; i < kAppBatch; ++i) {
            const int h = h0 + i * nsub;
            if (h >= heads) break;
            if (turns && h < a.Hq + a.Hkv) {
              uint32_t* wa = reinterpret_cast<uint32_t*>(&xa[i]);
              uint32_t* wb = reinterpret_cast<uint32_t*>(&xb[i]);
              auto up = [](uint32_t w) {
                return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
              };
              auto down = [](float x, float y) {
                const __nv_bfloat162 r = __floats2bfloat162_rn(x, y);
                return *reinterpret_cast<const uint32_t*>(&r);
              };
              if (INTERLEAVED) {                 // word j of a vector is one pair
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float2 p = up(wa[j]), r = up(wb[j]);
                  wa[j] = down(p.x * cs[j] - p.y * sn[j], p.y * cs[j] + p.x * sn[j]);
                  wb[j] = down(r.x * cs[j + 4] - r.y * sn[j + 4],
                               r.y * cs[j + 4] + r.x * sn[j + 4]);
                }
              } else {                           // channel j of the two vectors is one pair
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float2 x = up(wa[j]), y = up(wb[j]);
                  wa[j] = down(x.x * cs[2 * j] - y.x * sn[2 * j],
                               x.y * cs[2 * j + 1] - y.y * sn[2 * j + 1]);
                  wb[j] = down(y.x * cs[2 * j] + x.x * sn[2 * j],
                               y.y * cs[2 * j + 1] + x.y * sn[2 * j + 1]);
                }
              }
            }
            auto put = [&](__nv_bfloat16* dst) {
              *reinterpret_cast<uint4*>(dst + oa) = xa[i];
              *reinterpret_cast<uint4*>(dst + ob) = xb[i];
            };
            if (h < a.Hq) {
              put(a.q_out + (static_cast<size_t>(t) * a.Hq + h) * D);
              if (ring) {
                const size_t r = static_cast<size_t>(b) * 2 * a.ring_w + slot % a.ring_w;
                put(a.q_ring + (r * a.Hq + h) * D);
                put(a.q_ring + ((r + a.ring_w) * a.Hq + h) * D);
              }
            } else if (h < a.Hq + a.Hkv) {
              const int g = h - a.Hq;
              if (blk >= 0) put(a.k_cache + cache_row + static_cast<size_t>(g) * D);
              if (a.k_out != nullptr) put(a.k_out + (static_cast<size_t>(t) * a.Hkv + g) * D);
            } else if (blk >= 0) {
              put(a.v_cache + cache_row + static_cast<size_t>(h - a.Hq - a.Hkv) * D);
            }
          }
        }
      }
      if (a.bounds != nullptr && blk >= 0 && s_hi == page * 16 + 16) {
        __syncthreads();                         // the block's keys are in the page
        for (int i = threadIdx.x; i < a.Hkv * (D / 8); i += kAppThreads)
          page_bounds_unit(a.k_cache, a.bounds, blk, a.Hkv, D, i);
      }
    }
    base += total;
  }
}

constexpr int kBndThreads = 256;
constexpr int kBndPages = 8;      // pages per work item

struct BoundsArgs {
  const __nv_bfloat16* k_cache;
  __nv_bfloat16* bounds;
  const int32_t* block_table;
  const int32_t* ctx_len;
  const int32_t* from_slot;       // [B] or null
  int32_t* status;
  int B, Hkv, D, max_blocks, num_blocks, new_slots;
};

// Bounds of the complete pages of every sequence that hold a slot >= from_slot. A thread reads
// the 16 rows of 8 channels at once (256 bytes in flight); a page's rows are contiguous over
// the KV heads, so warps read whole lines.
__global__ void __launch_bounds__(kBndThreads) page_bounds_kernel(const BoundsArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ RowItems<kBndThreads> items;
  const int units = a.Hkv * (a.D / 8);
  // complete pages [first, last) of sequence b
  auto range = [&](int b, int& first) -> int {
    const int n_raw = a.ctx_len[b];
    const int64_t n = static_cast<int64_t>(n_raw) + a.new_slots;
    first = 0;
    if (n_raw < 0 || n > static_cast<int64_t>(a.max_blocks) * 16) {
      report(a.status, KARA_ERR_INVALID_ARG);
      return 0;
    }
    if (a.from_slot != nullptr) first = max(a.from_slot[b], 0) / 16;
    return max(static_cast<int>(n / 16) - first, 0);
  };
  int64_t base = 0;
  for (int b0 = 0; b0 < a.B; b0 += kBndThreads) {
    const int bt = b0 + static_cast<int>(threadIdx.x);
    int first, count = 0;
    if (bt < a.B) count = (range(bt, first) + kBndPages - 1) / kBndPages;
    row_items_scan(items, count);
    const int total = items.start[kBndThreads];
    const int64_t skip = base <= static_cast<int64_t>(blockIdx.x)
                             ? static_cast<int64_t>(blockIdx.x) - base
                             : (gridDim.x - (base - blockIdx.x) % gridDim.x) % gridDim.x;
    for (int64_t it = skip; it < total; it += gridDim.x) {
      const int row = row_items_find(items, static_cast<int>(it));
      const int b = b0 + row;
      const int pages = range(b, first);
      const int p0 = (static_cast<int>(it) - items.start[row]) * kBndPages;
      const int np = min(kBndPages, pages - p0);
      const int32_t* table = a.block_table + static_cast<size_t>(b) * a.max_blocks + first + p0;
      for (int i = threadIdx.x; i < np * units; i += kBndThreads) {
        const int p = i / units;
        const int blk = table[p];
        if (blk < 0 || blk >= a.num_blocks) {
          report(a.status, KARA_ERR_BAD_BLOCK);
          continue;
        }
        page_bounds_unit(a.k_cache, a.bounds, blk, a.Hkv, a.D, i - p * units);
      }
    }
    base += total;
  }
}

}  // namespace

kara_status launch_rope_append(const RopeAppendLaunch& L, cudaStream_t stream) {
  AppendArgs a;
  a.q = static_cast<const __nv_bfloat16*>(L.q);
  a.k = static_cast<const __nv_bfloat16*>(L.k);
  a.v = static_cast<const __nv_bfloat16*>(L.v);
  a.q_stride = L.q_stride;
  a.k_stride = L.k_stride;
  a.v_stride = L.v_stride;
  a.cu = L.cu_tokens;
  a.positions = L.positions;
  a.inv_freq = L.inv_freq;
  a.k_cache = static_cast<__nv_bfloat16*>(L.k_cache);
  a.v_cache = static_cast<__nv_bfloat16*>(L.v_cache);
  a.bounds = static_cast<__nv_bfloat16*>(L.bounds);
  a.q_ring = static_cast<__nv_bfloat16*>(L.q_ring);
  a.q_out = static_cast<__nv_bfloat16*>(L.q_out);
  a.k_out = static_cast<__nv_bfloat16*>(L.k_out);
  a.block_table = L.block_table;
  a.ctx_len = L.ctx_len;
  a.status = L.status;
  a.T = L.T;
  a.B = L.B;
  a.Hq = L.Hq;
  a.Hkv = L.Hkv;
  a.max_blocks = L.max_blocks;
  a.num_blocks = L.num_blocks;
  a.rd = L.rotary_dim;
  a.ring_w = L.ring_w;
  // n tokens of one sequence touch at most (n + 14) / 16 + 1 pages, and at most n
  const int64_t most = (static_cast<int64_t>(L.T) + 30 * static_cast<int64_t>(L.B)) / 16 + 1;
  const int grid = static_cast<int>(most < L.T ? most : L.T);
  if (L.D == 128) {
    if (L.interleaved)
      launch_pdl(rope_append_kernel<128, true>, dim3(grid), dim3(kAppThreads), 0, stream, a);
    else
      launch_pdl(rope_append_kernel<128, false>, dim3(grid), dim3(kAppThreads), 0, stream, a);
  } else {
    if (L.interleaved)
      launch_pdl(rope_append_kernel<64, true>, dim3(grid), dim3(kAppThreads), 0, stream, a);
    else
      launch_pdl(rope_append_kernel<64, false>, dim3(grid), dim3(kAppThreads), 0, stream, a);
  }
  return check_launch("paged_rope_append");
}

kara_status launch_page_bounds(const PageBoundsLaunch& L, cudaStream_t stream) {
  BoundsArgs a;
  a.k_cache = static_cast<const __nv_bfloat16*>(L.k_cache);
  a.bounds = static_cast<__nv_bfloat16*>(L.bounds);
  a.block_table = L.block_table;
  a.ctx_len = L.ctx_len;
  a.from_slot = L.from_slot;
  a.status = L.status;
  a.B = L.B;
  a.Hkv = L.Hkv;
  a.D = L.D;
  a.max_blocks = L.max_blocks;
  a.num_blocks = L.num_blocks;
  a.new_slots = L.new_slots;
  const int64_t most = static_cast<int64_t>(L.B) * ((L.max_blocks + kBndPages - 1) / kBndPages);
  int sms = 148;
  const int dev = device_slot();
  if (dev >= 0) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t wave = static_cast<int64_t>(sms) * 4;
  launch_pdl(page_bounds_kernel, dim3(static_cast<unsigned>(most < wave ? most : wave)),
             dim3(kBndThreads), 0, stream, a);
  return check_launch("paged_page_bounds");
}

}  // namespace kara
