// Streaming attention over chosen pages (block-sparse attention, and what rows that share a
// prefix have on their own), and the join of partial results.
//
// The products are those of the dense decode kernel: per page S^T = K Q^T and O^T += V^T P^T on
// warp-level m16n8k16 with the group's G <= 8 query heads as the 8-wide side, every K and V row
// of a KV head loaded once for the whole group through a per-warp ring of single pages. The
// work differs: the call's pages are one line per KV head, cut into equal ranges, and a warp
// carries (m, l, o) along its range as long as the row stays the same. All warps finish
// together whatever the rows' lengths, and a row leaves about as many partials as ranges touch
// it (128 rows of 128 selected pages and 4 KV heads on the 1776 warps of 148 SMs: fixed 8-page
// units would give the busiest warp 40 pages and a row 16 partials, ranges give 37 and 4 to 5).
// HBM-bound: that case reads its 537 MB in 95 to 98 us, 5.5 TB/s (84 % of measured). Taking ranges
// from a counter as warps become free (2 to 6 per warp) was 3 to 10 % slower than one each.
//
// The weights are rounded to bf16 for their product with V (at most 2^-8 of each), the type that
// the tensor cores take beside bf16 values and that of the dense decode kernel; the sums that divide
// the output are those of the unrounded weights, in fp32 as scores, maxima and outputs are.
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "page_mma.cuh"
#include "paged_plan.cuh"

namespace kara {

namespace {

constexpr int kStrThreads = 128;
constexpr int kStrWarps = 4;
constexpr int kStrBlocks = 3;        // resident blocks per SM (168 registers a thread)
constexpr int kStrUnit = 8;          // pages scored before their values are read
constexpr int kMaxSms = 160;         // workspaces are sized for this many

// The same bytes in flight for both head sizes: 16 KB per warp.
template <int D>
__host__ __device__ constexpr int str_stages() { return D == 128 ? 4 : 8; }
template <int D>
constexpr size_t str_smem_bytes() {
  return 1024 + static_cast<size_t>(kStrWarps) * str_stages<D>() * (page_bytes<D>() + 8);
}

struct StreamArgs {
  const __nv_bfloat16* q;
  const int32_t* block_table;
  const int32_t* sel;
  int sel_pages;
  StreamLine line;
  float* part_o;
  float2* part_ml;
  int32_t* status;
  int B, Hq, Hkv, max_blocks, num_blocks;
  float cs;                          // scale * log2(e)
};

// Up to kStrUnit pages of one row.
struct Piece {
  int i, row, n;       // list position, cache row, slots
  int e0, np;          // first page of the piece (LIST: list entry), pages
  bool ok;
};

// Walks the range [pos, end) of the line (warp-uniform; every lane calls it).
template <bool LIST>
struct RangeCursor {
  int pos, end, i, stop;     // stop: where row i ends on the line
  int4 r;
  __device__ __forceinline__ Piece next(const StreamArgs& a) {
    Piece x;
    x.ok = false;
    if (pos >= end) return x;
    if (pos >= stop) {
      // the last row that starts at or before pos, 32 candidates at a time
      const int lane = lane_id();
      int lo = 0, len = a.B;
      do {
        const int step = (len + 31) >> 5;
        const int off = lane * step;
        const int4 x = __ldcg(a.line.rows + lo + min(off, len - 1));
        const int hit = 31 - __clz(__ballot_sync(0xffffffffu, off < len && x.w <= pos));
        lo += hit * step;
        len = min(step, len - hit * step);
        r.x = __shfl_sync(0xffffffffu, x.x, hit);
        r.y = __shfl_sync(0xffffffffu, x.y, hit);
        r.z = __shfl_sync(0xffffffffu, x.z, hit);
        r.w = __shfl_sync(0xffffffffu, x.w, hit);
      } while (len > 1);
      i = lo;
      const int pages = (r.z + 15) / 16;
      stop = r.w + (LIST ? min(pages, a.sel_pages) : pages - r.y);
    }
    x.i = i;
    x.row = r.x;
    x.n = r.z;
    x.e0 = (LIST ? 0 : r.y) + pos - r.w;
    x.np = min(kStrUnit, min(stop, end) - pos);
    x.ok = x.np > 0;
    pos += x.np;
    return x;
  }
};

template <int D, int G, bool LIST>
__global__ void __launch_bounds__(kStrThreads, kStrBlocks)
page_stream_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const StreamArgs a) {
  static_assert(G <= 8, "at most 8 query heads per KV head");
  // The line was written before the kernel that this one follows: that one let it start only when
  // its own wait was over. LIST waits for it before the first list is read; otherwise the two run
  // side by side, and the wait comes at the end.
  bool waited = false;
  constexpr int kStages = str_stages<D>();
  constexpr int NCH = D / 64;                 // 64-channel chunks per row
  constexpr int KS = D / 16;                  // k-steps of S^T, m-tiles of O^T
  constexpr uint32_t kPage = page_bytes<D>();
  constexpr uint32_t kChunkBytes = 16 * 128;  // one 64-channel chunk of a page
  const int warp = warp_id(), lane = lane_id();
  const int grp = lane >> 2, tig = lane & 3;  // fragment row / column pair
  const int mtx = lane >> 3, mrow = lane & 7; // ldmatrix: lane feeds row mrow of matrix mtx

  extern __shared__ __align__(1024) uint8_t dsm[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* my_ring = ring + static_cast<size_t>(warp) * kStages * kPage;
  uint64_t* my_bars = reinterpret_cast<uint64_t*>(ring + kStrWarps * kStages * kPage) +
                      warp * kStages;
  const uint32_t ring_u32 = smem_u32(my_ring);
  if (lane == 0) {
    for (int st = 0; st < kStages; ++st) mbar_init(&my_bars[st], 1);
    fence_barrier_init();
  }
  __syncthreads();
  // the join may be scheduled now; it waits for this grid's results itself
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int total = __ldcg(a.line.total);
  const int R = stream_ranges(a.line, total);
  // neighbouring warps take the KV heads of the same pages, whose rows lie side by side in HBM
  const long long jobs = static_cast<long long>(R) * a.Hkv;
  const bool elected = elect_one();
  int issued = 0, done = 0;
  uint32_t phase = 0;      // parity bit per stage
  uint32_t pending = 0;    // stages with a load issued and not yet consumed
  bool aborted = false;
  for (long long job = static_cast<long long>(blockIdx.x) * kStrWarps + warp;
       job < jobs && !aborted; job += static_cast<long long>(gridDim.x) * kStrWarps) {
    const int range = static_cast<int>(job / a.Hkv), g = static_cast<int>(job % a.Hkv);
    RangeCursor<LIST> cursor;
    cursor.pos = range_start(range, R, total);
    cursor.end = range_start(range + 1, R, total);
    cursor.stop = cursor.pos;
    Piece cu = cursor.next(a);
    Piece nu = cursor.next(a);

    // LIST: lane j keeps the page number of the piece's entry j
    auto load_pages = [&](const Piece& x) -> int {
      if (!LIST || !x.ok || lane >= x.np) return 0;
      const int p = a.sel[(static_cast<size_t>(x.row) * a.Hkv + g) * a.sel_pages + x.e0 + lane];
      return min(max(p, 0), a.max_blocks - 1);
    };
    auto load_ids = [&](const Piece& x, int page) -> int {
      if (!x.ok || lane >= x.np) return -1;
      int blk = a.block_table[static_cast<size_t>(x.row) * a.max_blocks +
                              (LIST ? page : x.e0 + lane)];
      if (blk < 0 || blk >= a.num_blocks) {
        report(a.status, KARA_ERR_BAD_BLOCK);
        blk = -1;
      }
      return blk;
    };
    // B fragments of Q^T (column grp = query head g*G + grp when grp < G, else 0)
    auto load_q = [&](const Piece& x, uint32_t (&qb)[KS][2]) {
      const bool row_ok = x.ok && grp < G;
      const uint32_t* qrow = reinterpret_cast<const uint32_t*>(
          a.q + (static_cast<size_t>(x.ok ? x.row : 0) * a.Hq + g * G + (row_ok ? grp : 0)) * D);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qb[ks][0] = row_ok ? qrow[ks * 8 + tig] : 0u;
        qb[ks][1] = row_ok ? qrow[ks * 8 + 4 + tig] : 0u;
      }
    };
    uint32_t qb[KS][2];
    load_q(cu, qb);
    if (LIST && !waited) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      waited = true;
    }
    int pages_cu = load_pages(cu), pages_nu = load_pages(nu);
    int ids_cu = load_ids(cu, pages_cu), ids_nu = load_ids(nu, pages_nu);

    // Stream entries: a piece contributes 2 * np entries, K pages then V pages.
    int ustart = issued;     // stream index of cu's first entry
    volatile int no_abort = 0;
    auto top_up = [&]() {
      const int avail = ustart + 2 * cu.np + (nu.ok ? 2 * nu.np : 0);
      while (issued < done + kStages && issued < avail) {
        const int e = issued - ustart;
        const bool in_cu = e < 2 * cu.np;
        const int e2 = in_cu ? e : e - 2 * cu.np;
        const int npx = in_cu ? cu.np : nu.np;
        const bool is_v = e2 >= npx;
        const int j = is_v ? e2 - npx : e2;
        const int blk = __shfl_sync(0xffffffffu, in_cu ? ids_cu : ids_nu, j & 31);
        const int st = issued % kStages;
        if (blk >= 0) pending |= 1u << st;
        if (elected && blk >= 0) {
          uint8_t* dst = my_ring + st * kPage;
          mbar_expect_tx(&my_bars[st], kPage);
          const CUtensorMap* tm = is_v ? &tm_v : &tm_k;
#pragma unroll
          for (int c = 0; c < NCH; ++c)
            tma_load_4d(dst + c * kChunkBytes, tm, &my_bars[st], c * 64, g, 0, blk);
        }
        __syncwarp();
        ++issued;
      }
    };
    // Consumes stream entry t: its shared address, or 0 when the page was skipped (bad block,
    // reported) or the wait gave up (sets aborted).
    auto acquire = [&](int t, int blk) -> uint32_t {
      top_up();
      done = t + 1;
      if (blk < 0) return 0u;
      const int st = t % kStages;
      if (!mbar_wait(&my_bars[st], (phase >> st) & 1, &no_abort, a.status)) {
        aborted = true;
        return 0u;
      }
      phase ^= 1u << st;
      pending &= ~(1u << st);
      return ring_u32 + st * kPage;
    };
    auto valid_slots = [&](int j) -> int {     // slots of the piece's page j that the row holds
      const int page = LIST ? __shfl_sync(0xffffffffu, pages_cu, j) : cu.e0 + j;
      return min(16, cu.n - page * 16);
    };

    // the row's running exponent base and sum (heads 2tig, 2tig + 1; the sum over this lane's
    // slots) and unnormalised output
    float rm0 = -INFINITY, rm1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[KS][4];
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;

    while (cu.ok) {
      // ---- K pages: S^T for every page of the piece ----
      float sc[kStrUnit][4];
#pragma unroll
      for (int j = 0; j < kStrUnit; ++j) {
        sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = -INFINITY;
        if (j < cu.np && !aborted) {
          const int blk = __shfl_sync(0xffffffffu, ids_cu, j);
          const uint32_t kst = acquire(ustart + j, blk);
          const int valid = valid_slots(j);
          if (kst != 0u) {
            // two independent accumulator chains (even / odd k-steps), added at the end
            float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              const int slot = (mtx & 1) * 8 + mrow;
              const int d0 = ks * 16 + (mtx >> 1) * 8;
              uint32_t ka[4];
              ldsm_x4(kst + (d0 >> 6) * kChunkBytes + sw128(slot, (d0 & 63) >> 3), ka);
              mma_16816(acc[ks & 1], ka, qb[ks][0], qb[ks][1]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[0][e] += acc[1][e];
            // acc: (slot grp, heads 2tig, 2tig+1), (slot grp+8, heads 2tig, 2tig+1)
            const bool lo_ok = grp < valid, hi_ok = grp + 8 < valid;
            sc[j][0] = lo_ok ? acc[0][0] * a.cs : -INFINITY;
            sc[j][1] = lo_ok ? acc[0][1] * a.cs : -INFINITY;
            sc[j][2] = hi_ok ? acc[0][2] * a.cs : -INFINITY;
            sc[j][3] = hi_ok ? acc[0][3] * a.cs : -INFINITY;
          }
          __syncwarp();
        }
      }
      if (aborted) break;
      // ---- the exponent base of the row so far ----
      float m0 = rm0, m1 = rm1;
#pragma unroll
      for (int j = 0; j < kStrUnit; ++j) {
        m0 = fmaxf(m0, fmaxf(sc[j][0], sc[j][2]));
        m1 = fmaxf(m1, fmaxf(sc[j][1], sc[j][3]));
      }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, off));
        m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, off));
      }
      const float b0 = m0 == -INFINITY ? 0.f : m0;   // a head with no valid slot: all P = 0
      const float b1 = m1 == -INFINITY ? 0.f : m1;
      const float f0 = ex2(rm0 - b0), f1 = ex2(rm1 - b1);   // 0 for a fresh row
      rm0 = m0;
      rm1 = m1;
      l0 *= f0;
      l1 *= f1;
      uint32_t pb[kStrUnit][2];   // P^T B fragments per page: slots 2tig.. and 8+2tig.., head grp
#pragma unroll
      for (int j = 0; j < kStrUnit; ++j) {
        const float p0 = ex2(sc[j][0] - b0), p1 = ex2(sc[j][1] - b1);
        const float p2 = ex2(sc[j][2] - b0), p3 = ex2(sc[j][3] - b1);
        l0 += p0 + p2;
        l1 += p1 + p3;
        pb[j][0] = movmatrix_trans(pack_bf16(p0, p1));
        pb[j][1] = movmatrix_trans(pack_bf16(p2, p3));
      }
      // ---- V pages: O^T += V^T P^T ----
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        o[mt][0] *= f0;
        o[mt][1] *= f1;
        o[mt][2] *= f0;
        o[mt][3] *= f1;
      }
#pragma unroll
      for (int j = 0; j < kStrUnit; ++j) {
        if (j < cu.np && !aborted) {
          const int blk = __shfl_sync(0xffffffffu, ids_cu, j);
          const uint32_t vst = acquire(ustart + cu.np + j, blk);
          const int valid = valid_slots(j);
          if (vst != 0u) {
            // slots past the context may hold any bits (even NaN); P is 0 there, V is zeroed
            const int s_lo = 2 * tig, s_hi = 8 + 2 * tig;
            const uint32_t mlo =
                (s_lo < valid ? 0xffffu : 0u) | (s_lo + 1 < valid ? 0xffff0000u : 0u);
            const uint32_t mhi =
                (s_hi < valid ? 0xffffu : 0u) | (s_hi + 1 < valid ? 0xffff0000u : 0u);
            const bool partial_page = valid < 16;
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
              const int slot = (mtx >> 1) * 8 + mrow;
              const int c0 = mt * 16 + (mtx & 1) * 8;
              uint32_t va[4];
              ldsm_x4_trans(vst + (c0 >> 6) * kChunkBytes + sw128(slot, (c0 & 63) >> 3), va);
              if (partial_page) {
                va[0] &= mlo;
                va[1] &= mlo;
                va[2] &= mhi;
                va[3] &= mhi;
              }
              mma_16816(o[mt], va, pb[j][0], pb[j][1]);
            }
          }
          __syncwarp();
        }
      }
      if (aborted) break;
      // ---- the row's partial, when the next piece is another row's or none ----
      if (!nu.ok || nu.i != cu.i) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          l0 += __shfl_xor_sync(0xffffffffu, l0, off);
          l1 += __shfl_xor_sync(0xffffffffu, l1, off);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int h = 2 * tig + e;
          if (h < G) {
            const size_t at = static_cast<size_t>(cu.i + range) * a.Hq + g * G + h;
            float* dst = a.part_o + at * D;
            if (grp == 0) a.part_ml[at] = make_float2(e == 0 ? rm0 : rm1, e == 0 ? l0 : l1);
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
              dst[mt * 16 + grp] = o[mt][e];
              dst[mt * 16 + 8 + grp] = o[mt][2 + e];
            }
          }
        }
        rm0 = rm1 = -INFINITY;
        l0 = l1 = 0.f;
        // the next row's factor is 0, which does not clear an infinity or NaN
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
        load_q(nu, qb);
      }
      ustart += 2 * cu.np;
      cu = nu;
      ids_cu = ids_nu;
      pages_cu = pages_nu;
      if (!cu.ok) break;
      nu = cursor.next(a);
      pages_nu = load_pages(nu);
      ids_nu = load_ids(nu, pages_nu);
    }
  }
  if (aborted) {
    // a wait gave up (reported): let this warp's loads still in flight land before exiting
    volatile int give_up = 0;
    for (int st = 0; st < kStages; ++st)
      if ((pending >> st) & 1u) mbar_wait(&my_bars[st], (phase >> st) & 1, &give_up, a.status);
  }
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Join of a row's partials (m, l, o), base 2:
//     m = max m_i,  l = sum 2^(m_i - m) l_i,  out = sum 2^(m_i - m) o_i / l.
// A partial is empty where its l is 0, not where its m is -inf: scores that are all NaN leave no
// maximum, and their l and o are NaN.
// SHARE warps per (list position, query head) take its partials in turn, each with a batch of them
// in flight and a running (m, l, o) of its own, so that a partial is read once and without waiting
// for the maximum; a lane owns D / 32 channels. One warp each where the heads alone fill the SMs
// (3584 heads 153 -> 149 us and 144 -> 139.5 us for their calls), else four (896 heads 35.9 -> 34.4,
// 32 heads of 64 partials 30.2 -> 25.3).
constexpr int kJoinWarps = 4;        // per block
constexpr unsigned kJoinMany = 2048;

struct JoinArgs {
  StreamLine line;
  const float* part_o;
  const float2* part_ml;
  const PrefixHead* head;
  const PrefixGroup* groups;
  const int* row_group;
  const float* pre_o;
  const float2* pre_ml;
  __nv_bfloat16* out;
  int B, Hq, Hkv, G;
};

template <int D, int SHARE>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const JoinArgs a) {
  constexpr int V = D / 32;
  constexpr int kBatch = SHARE == 1 ? 8 : 4;
  __shared__ float red_o[kJoinWarps][D];
  __shared__ float red_m[kJoinWarps], red_l[kJoinWarps];
  const int lane = lane_id(), warp = warp_id() % SHARE;
  const int head = static_cast<int>(blockIdx.x) * (kJoinWarps / SHARE) + warp_id() / SHARE;
  const int i = head / a.Hq, h = head - i * a.Hq;
  if (i >= a.B) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int4 rw = a.line.rows[i];
  const int next = i + 1 < a.B ? a.line.rows[i + 1].w : -1;
  const int total = *a.line.total;
  if (rw.x < 0) {                                // not in a group: its output stays as it was
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int len = (next < 0 ? total : next) - rw.w;
  int r0 = 0, ntail = 0;
  if (len > 0) {
    const int R = stream_ranges(a.line, total);
    r0 = range_of(rw.w, R, total);
    ntail = range_of(rw.w + len - 1, R, total) - r0 + 1;
  }
  // the row's item among the shared ones and the blocks c0 .. c0 + npre - 1 that worked on it
  int npre = 0;
  long long row = 0;
  if (a.head != nullptr) {
    const PrefixGroup gr = a.groups[a.row_group[i]];
    if (gr.ktiles > 0) {
      const int g = h / a.G;
      const int qr = (i - gr.first) * a.G + h - g * a.G;
      const int t = qr / gr.item_rows, r = qr - t * gr.item_rows;
      const int rows_t = min(gr.item_rows, gr.rows * a.G - t * gr.item_rows);
      // the item's first key is unit a0 of the line
      const long long a0 = gr.flat + kItemCost +
                           static_cast<long long>(t * a.Hkv + g) * (gr.ktiles + kItemCost);
      const long long work = a.head->total;
      const int ctas = a.head->ctas;
      const int c0 = part_of(a0, ctas, work);
      npre = part_of(a0 + gr.ktiles - 1, ctas, work) - c0 + 1;
      row = static_cast<long long>(a.Hq) * gr.first +
            static_cast<long long>(t) * gr.item_rows * a.Hkv + static_cast<long long>(g) * rows_t +
            r + static_cast<long long>(kItemRows) * c0;
    }
  }
  const int parts = npre + ntail;
  // the line and the plan were written before the kernel that this one follows was let start
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float m = -INFINITY, l = 0.f, acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  for (int p0 = warp; p0 < parts; p0 += SHARE * kBatch) {
    float x[kBatch][V];
    float2 ml[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int p = p0 + e * SHARE;
      ml[e] = make_float2(-INFINITY, 0.f);
      if (p < parts) {
        const size_t at = p < npre ? static_cast<size_t>(row + static_cast<long long>(kItemRows) * p)
                                   : static_cast<size_t>(i + r0 + p - npre) * a.Hq + h;
        ml[e] = p < npre ? a.pre_ml[at] : a.part_ml[at];
        const float* src = (p < npre ? a.pre_o : a.part_o) + at * D + lane * V;
        if constexpr (V == 4)
          *reinterpret_cast<float4*>(x[e]) = *reinterpret_cast<const float4*>(src);
        else
          *reinterpret_cast<float2*>(x[e]) = *reinterpret_cast<const float2*>(src);
      }
    }
    float top = m;
#pragma unroll
    for (int e = 0; e < kBatch; ++e) top = fmaxf(top, ml[e].x);
    const float base = top == -INFINITY ? 0.f : top;
    const float f = ex2(m - base);
    m = top;
    l *= f;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= f;
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      if (ml[e].y == 0.f) continue;              // nothing in it (or none: o was not read)
      const float w = ex2(ml[e].x - base);
      l += w * ml[e].y;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(w, x[e][v], acc[v]);
    }
  }
  __nv_bfloat16* out = a.out + (static_cast<size_t>(rw.x) * a.Hq + h) * D;
  if constexpr (SHARE == 1) {
    const float inv = l == 0.f ? 0.f : 1.f / l;      // NaN stays NaN
#pragma unroll
    for (int v = 0; v < V; v += 2)
      *reinterpret_cast<__nv_bfloat162*>(out + lane * V + v) =
          __floats2bfloat162_rn(acc[v] * inv, acc[v + 1] * inv);
    return;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) red_o[warp][lane * V + v] = acc[v];
  if (lane == 0) {
    red_m[warp] = m;
    red_l[warp] = l;
  }
  __syncthreads();
  const int c = 2 * static_cast<int>(threadIdx.x);
  if (c >= D) return;
  float top = red_m[0];
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) top = fmaxf(top, red_m[w]);
  if (top == -INFINITY) top = 0.f;
  float sum = 0.f, r0o = 0.f, r1o = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    if (red_l[w] == 0.f) continue;
    const float f = ex2(red_m[w] - top);
    sum += f * red_l[w];
    r0o = fmaf(f, red_o[w][c], r0o);
    r1o = fmaf(f, red_o[w][c + 1], r1o);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<__nv_bfloat162*>(out + c) = __floats2bfloat162_rn(r0o * inv, r1o * inv);
}

template <int D, int G, bool LIST>
kara_status launch_dg(StreamLaunch* L, StreamArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                      cudaStream_t stream) {
  constexpr size_t smem = str_smem_bytes<D>();
  static std::atomic<int> per_sm[kMaxDevices];   // resident blocks per SM, queried once per device
  const int dev = device_slot();
  if (dev < 0) {
    set_last_error("paged attention", "no usable current CUDA device");
    return KARA_ERR_CUDA;
  }
  if (per_sm[dev].load() == 0) {
    cudaFuncSetAttribute(page_stream_kernel<D, G, LIST>,
                         cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    int n = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, page_stream_kernel<D, G, LIST>, kStrThreads,
                                                  smem);
    per_sm[dev].store(std::max(1, std::min(n, kStrBlocks)));
  }
  int sms = 148;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int blocks = per_sm[dev].load() * std::min(sms, kMaxSms);
  a.line.max_ranges = std::max(1, blocks * kStrWarps / L->Hkv);
  L->line.max_ranges = a.line.max_ranges;
  launch_pdl(page_stream_kernel<D, G, LIST>, dim3(static_cast<unsigned>(blocks)),
             dim3(kStrThreads), smem, stream, tk, tv, a);
  return check_launch("paged attention");
}

template <int D, bool LIST>
kara_status launch_d(StreamLaunch* L, StreamArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t stream) {
  switch (L->Hq / L->Hkv) {
    case 1: return launch_dg<D, 1, LIST>(L, a, tk, tv, stream);
    case 2: return launch_dg<D, 2, LIST>(L, a, tk, tv, stream);
    case 3: return launch_dg<D, 3, LIST>(L, a, tk, tv, stream);
    case 4: return launch_dg<D, 4, LIST>(L, a, tk, tv, stream);
    case 5: return launch_dg<D, 5, LIST>(L, a, tk, tv, stream);
    case 6: return launch_dg<D, 6, LIST>(L, a, tk, tv, stream);
    case 7: return launch_dg<D, 7, LIST>(L, a, tk, tv, stream);
    case 8: return launch_dg<D, 8, LIST>(L, a, tk, tv, stream);
    default: return KARA_ERR_UNSUPPORTED;
  }
}

}  // namespace

int stream_max_ranges(int hkv) {
  return std::max(1, kStrBlocks * kMaxSms * kStrWarps / hkv);
}

kara_status launch_stream(StreamLaunch* L, cudaStream_t stream) {
  StreamArgs a;
  a.q = static_cast<const __nv_bfloat16*>(L->q);
  a.block_table = L->block_table;
  a.sel = L->sel;
  a.sel_pages = L->sel_pages;
  a.line = L->line;
  a.part_o = L->part_o;
  a.part_ml = L->part_ml;
  a.status = L->status;
  a.B = L->B;
  a.Hq = L->Hq;
  a.Hkv = L->Hkv;
  a.max_blocks = L->max_blocks;
  a.num_blocks = L->num_blocks;
  a.cs = L->scale * 1.4426950408889634f;
  // paged pools as 4-D maps {d, Hkv, 16 slots, blocks}; box = one page of one KV head, 64
  // channels wide, 128-byte swizzle (the same map shape the dense decode kernel uses)
  const uint64_t dims[4] = {static_cast<uint64_t>(L->D), static_cast<uint64_t>(L->Hkv), 16,
                            static_cast<uint64_t>(L->num_blocks)};
  const uint64_t strides[3] = {static_cast<uint64_t>(L->D) * 2,
                               static_cast<uint64_t>(L->Hkv) * L->D * 2,
                               static_cast<uint64_t>(16) * L->Hkv * L->D * 2};
  CUtensorMap tk, tv;
  if (!make_bf16_map_4d(&tk, L->k_cache, dims, strides, 16) ||
      !make_bf16_map_4d(&tv, L->v_cache, dims, strides, 16))
    return KARA_ERR_CUDA;
  const bool list = !L->beside;
  if (L->D == 128)
    return list ? launch_d<128, true>(L, a, tk, tv, stream)
                : launch_d<128, false>(L, a, tk, tv, stream);
  if (L->D == 64)
    return list ? launch_d<64, true>(L, a, tk, tv, stream)
                : launch_d<64, false>(L, a, tk, tv, stream);
  return KARA_ERR_UNSUPPORTED;
}

kara_status launch_join(const JoinLaunch& L, cudaStream_t stream) {
  JoinArgs a;
  a.line = L.line;
  a.part_o = L.part_o;
  a.part_ml = L.part_ml;
  a.head = L.head;
  a.groups = L.groups;
  a.row_group = L.row_group;
  a.pre_o = L.pre_o;
  a.pre_ml = L.pre_ml;
  a.out = static_cast<__nv_bfloat16*>(L.out);
  a.B = L.B;
  a.Hq = L.Hq;
  a.Hkv = L.Hkv;
  a.G = L.Hq / L.Hkv;
  const unsigned heads = static_cast<unsigned>(L.B) * static_cast<unsigned>(L.Hq);
  const dim3 block(32 * kJoinWarps);
  if (heads >= kJoinMany) {
    const dim3 grid((heads + kJoinWarps - 1) / kJoinWarps);
    if (L.D == 128) launch_pdl(join_kernel<128, 1>, grid, block, 0, stream, a);
    else launch_pdl(join_kernel<64, 1>, grid, block, 0, stream, a);
  } else {
    if (L.D == 128) launch_pdl(join_kernel<128, 4>, dim3(heads), block, 0, stream, a);
    else launch_pdl(join_kernel<64, 4>, dim3(heads), block, 0, stream, a);
  }
  return check_launch("paged attention");
}

}  // namespace kara
