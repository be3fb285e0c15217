// Decode attention of rows that share their first pages (paged_prefix_attn): N sequences
// behind one prompt, or many samples of it, read the shared K and V once for all.
//
// For a group of N rows with a prefix of P pages, the N * G queries of a KV head form one
// matrix: S = Q K^T and O += P V on tcgen05 with 128 keys per step, so a byte of the prefix
// serves N * G queries instead of G. Every row's own slots behind the prefix go through the
// streaming decode kernel. Softmax statistics are base 2 and partial results (m, l, o), which
// join at the end:
//     m = max m_i,  l = sum 2^(m_i - m) l_i,  out = sum 2^(m_i - m) o_i / l.
// The weights P are rounded to bf16 (at most 2^-8 of each), the type that the tensor cores take
// beside bf16 values; l sums the unrounded ones in fp32.
// Four kernels: plan (groups, rows, the prefix work in units of 128 keys), prefix, stream (the rows'
// own pages, beside the prefix kernel), join.
//
// The prefix work of all groups, tiles of 256 queries and KV heads is one line of key tiles,
// cut into equal parts, one per block: all blocks finish together whatever the groups' sizes,
// and an item (group, query tile, KV head) that spans several parts leaves one partial in each.
#include <cuda.h>

#include <cstdint>
#include <limits>

#include "common.cuh"
#include "internal.h"
#include "paged_plan.cuh"
#include "row_items.cuh"

namespace kara {

namespace {

constexpr int kKeys = 128;              // keys per step
constexpr int kTilePages = kKeys / 16;
constexpr int kPart = 96;               // keys whose weights are handed over first (64: 0.5 % slower)
constexpr int kRows = 128;              // query rows per tensor-core tile
static_assert(kItemRows == 2 * kRows, "one tensor-core tile per softmax team");
constexpr int kMaxCtas = 160;           // grid limit (workspace rows are sized by it)
// Small calls spread over as many blocks and warps as there are tiles and page pairs: their time is
// the longest chain (eight rows behind 1K slots 24 us with 8 blocks, 18 with 44; 17.5 with 4 own
// pages per warp, 16.5 with 2).
constexpr int kMinTiles = 1;            // key tiles that are worth a block
constexpr int kTailMinPages = 2;        // a row's own pages that are worth a warp

struct PrefixArgs {
  const __nv_bfloat16* q;
  const int32_t* block_table;
  const int32_t* ctx_len;
  const int32_t* group_ptr;
  const int32_t* group_rows;     // or null: list position = cache row
  const int32_t* prefix_pages;
  PrefixHead* head;
  PrefixGroup* groups;
  int4* rows;                    // [B]: the streaming kernel's line
  int* row_group;                // [B]
  float* part_o;                 // prefix partials: [Hq B + 256 ctas, D]
  float2* part_ml;
  int32_t* status;
  int B, Hq, Hkv, G, max_blocks, num_blocks, num_groups, extra, ctas;
  float cs;                      // |scale| * log2(e)
  int negate;                    // scale < 0: the queries' signs are flipped
};

constexpr int kPlanThreads = 256;

// One block. A group of one row has nothing to share: its pages are all its own.
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PrefixArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // few groups stay in shared memory: the rows' searches would wait for L2 at every step
  constexpr int kNear = kPlanThreads;
  __shared__ RowItems<kPlanThreads> items;
  __shared__ PrefixGroup near_groups[kNear];
  __shared__ int near_ptr[kNear];
  const bool near = a.num_groups <= kNear;
  long long flat = 0;
  for (int j0 = 0; j0 < a.num_groups; j0 += kPlanThreads) {
    const int j = j0 + static_cast<int>(threadIdx.x);
    PrefixGroup gr = {};
    int len = 0;
    if (j < a.num_groups) {
      const int lo = a.group_ptr[j], hi = a.group_ptr[j + 1], pages = a.prefix_pages[j];
      // an empty group has no pages: what prefix_pages holds for it does not matter
      if (lo < 0 || hi < lo || hi > a.B || (hi > lo && (pages < 0 || pages > a.max_blocks))) {
        report(a.status, KARA_ERR_INVALID_ARG);
      } else if (hi > lo) {
        gr.first = lo;
        gr.rows = hi - lo;
        gr.pages = pages;
        gr.row0 = a.group_rows != nullptr ? a.group_rows[lo] : lo;
        if (gr.row0 < 0 || gr.row0 >= a.B) {
          report(a.status, KARA_ERR_INVALID_ARG);
          gr.rows = 0;
        } else if (gr.rows > 1) {
          gr.ktiles = (pages + kTilePages - 1) / kTilePages;
          // even items: their blocks take the same time per key tile
          const int q = gr.rows * a.G, items_q = (q + kItemRows - 1) / kItemRows;
          gr.item_rows = (q + items_q - 1) / items_q;
          len = gr.ktiles == 0 ? 0 : items_q * a.Hkv * (gr.ktiles + kItemCost);
        }
      }
    }
    row_items_scan(items, len);
    if (j < a.num_groups) {
      gr.flat = flat + items.start[threadIdx.x];
      a.groups[j] = gr;
      if (near) {
        near_groups[j] = gr;
        near_ptr[j] = a.group_ptr[j];
      }
    }
    flat += items.start[kPlanThreads];
  }
  if (threadIdx.x == 0) {
    const long long most = flat / kMinTiles;
    a.head->total = flat;
    a.head->ctas = static_cast<int>(most < 1 ? 1 : most < a.ctas ? most : a.ctas);
  }
  __syncthreads();               // the groups are written
  int line = 0;
  for (int i0 = 0; i0 < a.B; i0 += kPlanThreads) {
    const int i = i0 + static_cast<int>(threadIdx.x);
    int4 r = make_int4(-1, 0, 0, 0);
    int mine = 0;
    if (i < a.B) {
      int lo = 0, hi = a.num_groups;             // ptr[lo] <= i < ptr[hi] where there is one
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((near ? near_ptr[mid] : a.group_ptr[mid]) <= i) lo = mid;
        else hi = mid;
      }
      a.row_group[i] = lo;
      const PrefixGroup gr = near ? near_groups[lo] : a.groups[lo];
      if (i >= gr.first && i < gr.first + gr.rows) {
        const int row = a.group_rows != nullptr ? a.group_rows[i] : i;
        if (row < 0 || row >= a.B) {
          report(a.status, KARA_ERR_INVALID_ARG);
        } else {
          const int n = a.ctx_len[row];
          const long long len = static_cast<long long>(n) + a.extra;
          const long long most = static_cast<long long>(a.max_blocks) * 16;
          if (n < 0 || len < static_cast<long long>(gr.pages) * 16 || len > most)
            report(a.status, KARA_ERR_INVALID_ARG);
          r.x = row;
          r.y = gr.rows > 1 ? gr.pages : 0;
          r.z = static_cast<int>(len < 0 ? 0 : len > most ? most : len);
          mine = max((r.z + 15) / 16 - r.y, 0);
        }
      }
    }
    row_items_scan(items, mine);
    r.w = line + items.start[threadIdx.x];
    if (i < a.B) a.rows[i] = r;
    line += items.start[kPlanThreads];
  }
  if (threadIdx.x == 0) a.head->tail_pages = line;
}

// Items of up to kRows query rows go to team 0 alone, larger ones half to each team.
__device__ __forceinline__ int team0_rows(int rows) { return rows > kRows ? (rows + 1) / 2 : rows; }

// Warp-wide wait: every lane calls it and gets the same answer. Bounded (about 1.6 s at boost
// clock) and short: the hot loops have to stay in the instruction cache (with 82 KB of code one
// fetch in twenty missed it and tiles took twice as long). A wait that gives up raises *abort,
// which the block reports when it leaves.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const uint32_t t0 = static_cast<uint32_t>(clock());
#pragma unroll 1
    do {
      ok = mbar_try_wait(bar, parity);
    } while (!ok && *abort == 0 && static_cast<uint32_t>(clock()) - t0 < 3000000000u);
    if (!ok) *abort = 1;
  }
  return __all_sync(0xffffffffu, ok) != 0;
}

// The part of an item that one block works on: key tiles [kt0, kt1).
struct Seg {
  int first, row0, pages, g, kt0, kt1, q0, rows;   // q0: first query row of the item in its group
  long long out_row;                               // first partial row
};

// Walks block c's part of the line of key tiles.
struct SegCursor {
  long long pos, end;
  int c, j;
  __device__ __forceinline__ void init(const PrefixArgs& a, int cta) {
    c = cta;
    const long long total = a.head->total;
    const int n = a.head->ctas;
    pos = end = 0;
    j = 0;
    if (cta >= n) return;
    pos = part_start(cta, n, total);
    end = part_start(cta + 1, n, total);
    int lo = 0, hi = a.num_groups;               // the last group with flat <= pos
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.groups[mid].flat <= pos) lo = mid;
      else hi = mid;
    }
    j = lo;
  }
  __device__ __forceinline__ bool next(const PrefixArgs& a, Seg& s) {
    while (true) {
    if (pos >= end) return false;
    PrefixGroup gr = a.groups[j];
    while (j + 1 < a.num_groups && a.groups[j + 1].flat <= pos) gr = a.groups[++j];
    const int cost = gr.ktiles + kItemCost;      // an item's first kItemCost units hold no keys
    const int local = static_cast<int>(pos - gr.flat);
    const int x = local / cost;
    const int t = x / a.Hkv;
    const int u0 = local - x * cost;
    const int u1 = static_cast<int>(min(static_cast<long long>(cost), u0 + (end - pos)));
    pos += u1 - u0;
    if (u1 <= kItemCost) continue;
    s.g = x - t * a.Hkv;
    s.kt0 = max(u0 - kItemCost, 0);
    s.kt1 = u1 - kItemCost;
    s.first = gr.first;
    s.row0 = gr.row0;
    s.pages = gr.pages;
    s.q0 = t * gr.item_rows;
    s.rows = min(gr.item_rows, gr.rows * a.G - s.q0);
    s.out_row = static_cast<long long>(a.Hq) * gr.first + static_cast<long long>(s.q0) * a.Hkv +
                static_cast<long long>(s.g) * s.rows + static_cast<long long>(kItemRows) * c;
    return true;
    }
  }
};

constexpr int kPfxThreads = 384;        // warp 0: TMA, warps 1-2: UMMA, warps 4-11: softmax teams
constexpr int kTeamThreads = 128;       // one thread per query row
constexpr int kRegsLow = 72, kRegsHigh = 208;   // registers a thread after the split
constexpr uint32_t kTmemS = 0;          // S of team w at 128 w; its P (bf16) over S's columns
constexpr uint32_t kTmemO = 256;        // O of team w at 256 + 128 w

template <int D>
struct PfxSmem {
  static constexpr int NCH = D / 64;
  static constexpr uint32_t kChunk = kKeys * 128;          // 64 channels of 128 rows
  static constexpr uint32_t kTile = NCH * kChunk;          // one K or V tile, one Q tile
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr uint32_t q_off = 0;
  static constexpr uint32_t kv_off = 2 * kTile;
  static constexpr uint32_t bar_off = kv_off + kStages * kTile;
  static constexpr int kBars = 2 * kStages + 2 + 3 + 4 + 2 + 2 + 8 + 1;
  static constexpr uint32_t bytes = bar_off + kBars * 8 + 16;
};

// The shared pages of all groups. Per key tile of 128 keys the products of 256 query rows take 2050
// cycles of the tensor cores (d = 128) and their exponentials 2050 of the exponential unit (moving a
// quarter of them to the FMA pipe changed nothing); K and V of the tile take 2800 cycles of an
// SM's share of HBM. So HBM bounds groups of up to about 128 query rows, products and exponentials larger ones,
// whose softmax and products alternate between two teams of 128 rows. Rows live in tensor memory:
// S and P of a row share columns, one thread owns the row, no statistics cross threads.
// Measured: 128 rows of 28 heads behind 32K slots 76 us, 0.79 PFLOP/s (48 % of measured); 16 groups
// of 3 to 15 rows of 32 heads behind 240 to 7.4K slots 48 us for 195 MB, 4.1 TB/s (62 %): an item of
// few rows is one team's, whose chain of load, maximum and exponentials is longer than the tile's
// share of HBM.
template <int D>
__global__ void __launch_bounds__(kPfxThreads, 1)
prefix_attn_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const PrefixArgs a) {
  using L = PfxSmem<D>;
  constexpr int NCH = L::NCH;
  constexpr int kStages = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* q_buf = smem + L::q_off;
  uint8_t* kv_buf = smem + L::kv_off;
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + L::bar_off);
  uint64_t* kv_empty = kv_full + kStages;
  uint64_t* q_full = kv_empty + kStages;      // [2] the team's queries are in shared memory
  uint64_t* s_full = q_full + 2;              // [3] S of team w; [2]: team 0's second buffer
  uint64_t* p_full = s_full + 3;              // [team][part]: P written, S read, O rescaled
  uint64_t* o_full = p_full + 4;              // [2] O += P V done
  uint64_t* drained = o_full + 2;
  uint64_t* turn = drained + 2;               // [team][quad]: the warp may exponentiate
  uint64_t* handover = turn + 8;              // one team's items after two teams', or before
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(handover + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 2);               // one arrival per issuer
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&q_full[w], kTeamThreads / 32);
      mbar_init(&s_full[w], 1);
      mbar_init(&p_full[2 * w], 4);
      mbar_init(&p_full[2 * w + 1], 4);
      mbar_init(&o_full[w], 1);
    }
    mbar_init(&s_full[2], 1);
    mbar_init(&drained[0], 1);
    mbar_init(&drained[1], 1);
    for (int i = 0; i < 8; ++i) mbar_init(&turn[i], 1);
    mbar_init(handover, 8);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  asm volatile("griddepcontrol.wait;" ::: "memory");   // the plan is written
  // the streaming kernel may start: it reads the plan only, and waits for this kernel at its end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  SegCursor cur;
  cur.init(a, blockIdx.x);
  Seg sg;

  // registers: four warps give up what the softmax warps take; the launch has checked that the
  // block was given that many
  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");   // kRegsLow
  if (warp == 0) {
    // ---- TMA producer: K(0), then K(i), V(i - 1), the order of use ----
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    int issued = 0;
    bool ok = true;
    const bool elected = elect_one();
    while (ok && cur.next(a, sg)) {
      const int32_t* table = a.block_table + static_cast<size_t>(sg.row0) * a.max_blocks;
      // pages past the prefix in its last tile: the block behind the pool, which a copy fills with
      // zeros (their weights are 0, and so are the values: 0 x inf would be NaN)
      auto block_of = [&](int kt) -> int {
        if (lane >= kTilePages) return 0;
        const int page = kt * kTilePages + lane;
        if (page >= sg.pages) return a.num_blocks;
        int blk = table[page];
        if (blk < 0 || blk >= a.num_blocks) {
          report(a.status, KARA_ERR_BAD_BLOCK);
          blk = 0;
        }
        return blk;
      };
      auto load = [&](const CUtensorMap* tm, int blk) -> bool {
        const int st = issued % kStages;
        if (!wait_warp(&kv_empty[st], ((issued / kStages) & 1) ^ 1, abort_flag))
          return false;
        if (elected) mbar_expect_tx(&kv_full[st], L::kTile);
#pragma unroll
        for (int p = 0; p < kTilePages; ++p) {
          const int id = __shfl_sync(0xffffffffu, blk, p);
          if (elected) {
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch)
              tma_load_4d(kv_buf + st * L::kTile + ch * L::kChunk + p * 2048, tm, &kv_full[st],
                          ch * 64, sg.g, 0, id);
          }
        }
        __syncwarp();
        ++issued;
        return true;
      };
      int blk = block_of(sg.kt0), blk_v = 0;
      for (int kt = sg.kt0; ok && kt <= sg.kt1; ++kt) {
        const int blk_next = kt + 1 < sg.kt1 ? block_of(kt + 1) : 0;
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
          const bool key = e == 0;
          if (ok && (key ? kt < sg.kt1 : kt > sg.kt0)) ok = load(key ? &tm_k : &tm_v, key ? blk : blk_v);
        }
        blk_v = blk;
        blk = blk_next;
      }
    }
    if (!ok) {
      // a wait gave up (reported): let the copies in flight land before the block leaves
      volatile int give_up = 0;
      for (int st = 0; st < kStages; ++st)
        if (issued > st)
          wait_warp(&kv_full[st], ((issued - 1 - st) / kStages) & 1, &give_up);
    }
  } else if (warp == 1 || warp == 2) {
    // ---- UMMA issuers, one per team. Step i of team w: O_w += P_w(i-1) V(i-1), then S_w(i) = Q_w
    // K(i)^T, which overwrites P_w(i-1) (a thread's products execute in the order of issue). The
    // teams' steps interleave: one team's products, and its issuer's waits (about 100 cycles
    // each, as long as two products), run while the other team exponentiates. One team alone:
    // S(i) goes to the buffers in turn, ahead of O += P(i-1) V(i-1), so that the team's next
    // tile is ready when it has finished one. The warp waits, an elected thread issues. ----
    constexpr uint32_t idesc_s = idesc_bf16_f32(kRows, kKeys);
    constexpr uint32_t idesc_o = idesc_bf16_f32(kRows, D) | (1u << 16);   // V is N-major
    const int w = warp - 1;
    const bool elected = elect_one();
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return wait_warp(bar, parity, abort_flag);
    };
    uint32_t q_ph = 0, p_ph = 0;
    int used = 0;                               // ring entries consumed
    bool ok = true;
    while (ok && cur.next(a, sg)) {
      const bool both = sg.rows > kRows;
      const bool on = w == 0 || both;
      const int n = sg.kt1 - sg.kt0;
      if (on) {
        ok = wait(&q_full[w], q_ph);
        q_ph ^= 1;
      }
      for (int i = 0; ok && i <= n; ++i) {
        const int k_at = used, v_at = used + (i < n ? 1 : 0);
        const int ks = k_at % kStages, vs = v_at % kStages;
        auto scores = [&]() -> bool {           // S = Q_w K(i)^T
          if (!wait(&kv_full[ks], (k_at / kStages) & 1)) return false;
          tc_fence_after();
          if (elected) {
            if (on) {
              const int buf = both ? w : i & 1;
              const uint32_t q_addr = smem_u32(q_buf + w * L::kTile);
              const uint32_t k_addr = smem_u32(kv_buf + ks * L::kTile);
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = (k >> 2) * L::kChunk + (k & 3) * 32;
                umma_bf16(tmem + kTmemS + buf * 128, sw128_kmajor_desc(q_addr + off),
                          sw128_kmajor_desc(k_addr + off), idesc_s, k > 0 ? 1u : 0u);
              }
              umma_commit(&s_full[both ? w : (i & 1) * 2]);
            }
            umma_commit(&kv_empty[ks]);
          }
          __syncwarp();
          return true;
        };
        auto weigh = [&]() -> bool {            // O_w += P(i-1) V(i-1)
          if (!wait(&kv_full[vs], (v_at / kStages) & 1)) return false;
          if (on) {
            const int buf = both ? w : (i - 1) & 1;
            const uint32_t v_addr = smem_u32(kv_buf + vs * L::kTile);
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              if (!wait(&p_full[2 * w + part], p_ph)) return false;
              tc_fence_after();
              if (elected) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k) {
                  if ((k < kPart / 16) != (part == 0)) continue;
                  umma_bf16_ts(tmem + kTmemO + w * 128, tmem + kTmemS + buf * 128 + k * 8,
                               sw128_mnmajor_desc(v_addr + k * 2048, L::kChunk, 1024), idesc_o,
                               (i > 1 || k > 0) ? 1u : 0u);
                }
                if (part == 1) umma_commit(&o_full[w]);
              }
              __syncwarp();
            }
            p_ph ^= 1;
          }
          if (elected) umma_commit(&kv_empty[vs]);
          __syncwarp();
          return true;
        };
#pragma unroll 1
        for (int e = 0; ok && e < 2; ++e) {
          if ((e == 0) != both) {
            if (i < n) ok = scores();
          } else {
            if (i > 0) ok = weigh();
          }
        }
        used += (i < n ? 1 : 0) + (i > 0 ? 1 : 0);
      }
    }
    if (!ok) {                                  // products in flight still read shared memory
      volatile int give_up = 0;
      if (elected) umma_commit(&drained[w]);
      __syncwarp();
      wait_warp(&drained[w], 0, &give_up);
    }
  } else if (warp >= 4) {
    // ---- softmax teams: a thread owns one query row (TMEM lane) and holds its 128 scores of a
    // key tile in registers ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");   // kRegsHigh
    const int w = (warp - 4) >> 2;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t o_col = lane_base + kTmemO + w * 128;
    uint8_t* q_tile = q_buf + w * L::kTile;
    const uint32_t flip = a.negate ? 0x80008000u : 0u;
    const float2 cs2 = make_float2(a.cs, a.cs);
    uint32_t s_ph[3] = {0, 0, 0}, o_ph = 0;   // o_ph: parity of the next product to complete
    uint32_t t_ph = w == 0 ? 1 : 0;           // team 0 goes first
    uint32_t h_ph = 0;
    int before = 0;                           // teams of the segment before (0: none)
    bool aborted = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!aborted) aborted = !wait_warp(bar, parity, abort_flag);
    };
    while (!aborted && cur.next(a, sg)) {
      const int rows0 = team0_rows(sg.rows);
      const int row0 = w == 0 ? 0 : rows0;      // the team's rows of the item
      const int live = w == 0 ? rows0 : sg.rows - rows0;
      const bool one_team = sg.rows <= kRows;
      // A team on its own also uses the other's S buffer. So where segments of one team and of two
      // follow each other, both teams finish what they have before either starts (its issuer
      // waits for the team's queries).
      const int teams = one_team ? 1 : 2;
      if (before != 0 && before != teams) {
        if (lane == 0) mbar_arrive(handover);
        wait(handover, h_ph);
        h_ph ^= 1;
        if (aborted) break;
      }
      before = teams;
      if (live <= 0) continue;
      const bool warp_on = quad * 32 < live;
      // the warp's 32 query rows into the swizzled tile, 16 bytes per lane, all in flight at once
      // (rows past the last: copies of it, whose results are not read)
      if (warp_on) {
        constexpr int kPer = D / 8;             // lanes per row
        constexpr int kTurns = kPer;            // 32 rows, 32 / kPer at a time
        const int gi = lane % kPer, r0 = quad * 32 + lane / kPer;
        const __nv_bfloat16* src[kTurns];
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
          const int r = r0 + t * (32 / kPer);
          const int qr = sg.q0 + row0 + min(r, live - 1);
          const int member = qr / a.G, h = qr - member * a.G;
          int b = sg.first + member;
          if (a.group_rows != nullptr) b = min(max(a.group_rows[b], 0), a.B - 1);   // reported
          src[t] = a.q + (static_cast<size_t>(b) * a.Hq + sg.g * a.G + h) * D + gi * 8;
        }
        uint4 x[kTurns];
#pragma unroll
        for (int t = 0; t < kTurns; ++t) x[t] = *reinterpret_cast<const uint4*>(src[t]);
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
          const int r = r0 + t * (32 / kPer);
          x[t].x ^= flip;
          x[t].y ^= flip;
          x[t].z ^= flip;
          x[t].w ^= flip;
          *reinterpret_cast<uint4*>(q_tile + (gi >> 3) * L::kChunk + (r >> 3) * 1024 +
                                    (r & 7) * 128 + (((gi & 7) ^ (r & 7)) << 4)) = x[t];
        }
        fence_proxy_async();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[w]);
      float m = -INFINITY, l = 0.f;             // m: the exponent base, in units of raw S
      const int n = sg.kt1 - sg.kt0;
      for (int i = 0; i < n; ++i) {
        const int buf = one_team ? i & 1 : w;
        const int bar = one_team ? (i & 1) * 2 : w;
        wait(&s_full[bar], s_ph[bar]);
        s_ph[bar] ^= 1;
        if (aborted) break;
        if (!warp_on) {
          // not before product i - 1: an arrival for step i must not count for the step before
          if (i > 0) {
            wait(&o_full[w], o_ph);
            o_ph ^= 1;
          }
          if (!one_team) {
            wait(&turn[w * 4 + quad], t_ph);
            t_ph ^= 1;
          }
          if (lane == 0) {
            if (!one_team) mbar_arrive(&turn[(w ^ 1) * 4 + quad]);
            mbar_arrive(&p_full[2 * w]);
            mbar_arrive(&p_full[2 * w + 1]);
          }
        } else {
          tc_fence_after();
          const uint32_t s_col = lane_base + kTmemS + buf * 128;
          const int valid = (sg.pages - (sg.kt0 + i) * kTilePages) * 16;
          if (valid < kKeys) {                  // pages past the prefix: their scores become -inf
#pragma unroll 1
            for (int c = valid; c < kKeys; c += 16) tmem_st16_fill(s_col + c, -INFINITY);
            tmem_wait_st();
          }
          float v[kKeys];
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) tmem_ld32(s_col + c, v + c);
          tmem_wait_ld();
          reg_fence<kKeys>(v);
          float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kKeys; e += 8) {
#pragma unroll
            for (int t = 0; t < 4; ++t) mq[t] = fmax3(mq[t], v[e + 2 * t], v[e + 2 * t + 1]);
          }
          const float mx = fmaxf(fmax3(mq[0], mq[1], mq[2]), mq[3]);
          // the base moves only when the row maximum outgrows it by 2^8 (or on the first tile):
          // weights up to 2^8 lose nothing in fp32 sums and floating bf16
          const bool move = i > 0 && (mx - m) * a.cs > 8.f;
          if (i == 0) m = mx;
          bool waited = i == 0;                 // for O += P V of step i - 1
          if (__any_sync(0xffffffffu, move)) {
            wait(&o_full[w], o_ph);             // O is complete up to step i - 1
            waited = true;
            if (aborted) break;
            tc_fence_after();
            const float to = move ? mx : m;
            const float f = to == m ? 1.f : ex2((m - to) * a.cs);
            m = to;
            l *= f;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float o[16];
              uint32_t u[16];
              tmem_ld16(o_col + c, o);
              tmem_wait_ld();
              reg_fence<16>(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * f);
              tmem_st16(o_col + c, u);
            }
          }
          // m - m: a base of +inf makes the whole row NaN, as it should be
          const float nb = m == -INFINITY ? 0.f : (m - m) - m * a.cs;
          const float2 nb2 = make_float2(nb, nb);
          // the two teams' warps of a scheduler exponentiate in turns: left to themselves they fall
          // into step, share the exponential unit and then both wait for their products
          if (!one_team) {
            wait(&turn[w * 4 + quad], t_ph);
            t_ph ^= 1;
            if (aborted) break;
          }
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            uint32_t u[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 x = ffma2(make_float2(v[c + e], v[c + e + 1]), cs2, nb2);
              const float2 p = make_float2(ex2(x.x), ex2(x.y));
              sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], p);
              const __nv_bfloat162 pb = __floats2bfloat162_rn(p.x, p.y);
              u[e / 2] = *reinterpret_cast<const uint32_t*>(&pb);
            }
            tmem_st16(s_col + c / 2, u);
            if (c == kPart - 32) {              // the product may start on the first keys
              if (!waited) wait(&o_full[w], o_ph);   // its phase: none is ever two behind
              waited = true;
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&p_full[2 * w]);
            }
          }
          sum[0] = fadd2(sum[0], sum[1]);
          l += sum[0].x + sum[0].y;
          if (!one_team && lane == 0) mbar_arrive(&turn[(w ^ 1) * 4 + quad]);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * w + 1]);
          if (i > 0) o_ph ^= 1;
          if (aborted) break;
        }
      }
      if (aborted) break;
      wait(&o_full[w], o_ph);
      o_ph ^= 1;
      if (aborted) break;
      if (warp_on) {
        tc_fence_after();
        const size_t r = static_cast<size_t>(sg.out_row) + row0 + row;
        if (row < live) a.part_ml[r] = make_float2(m * a.cs, l);
        float* dst = a.part_o + r * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float v[32];
          tmem_ld32(o_col + c, v);
          tmem_wait_ld();
          reg_fence<32>(v);
          if (row < live) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(dst + c + e) =
                  make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
        }
        tc_fence_before();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag != 0) report(a.status, KARA_ERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

size_t align_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct PrefixLayout {
  size_t head, groups, rows, row_group, part_o, part_ml, tail_o, tail_ml, total;
};
PrefixLayout prefix_layout(int B, int Hq, int Hkv, int D) {
  PrefixLayout l;
  const size_t part_rows = static_cast<size_t>(B) * Hq + static_cast<size_t>(kItemRows) * kMaxCtas;
  const size_t tail_rows = (static_cast<size_t>(B) + stream_max_ranges(Hkv)) * Hq;
  l.head = 0;
  l.groups = align_up(sizeof(PrefixHead));
  l.rows = align_up(l.groups + static_cast<size_t>(B) * sizeof(PrefixGroup));
  l.row_group = align_up(l.rows + static_cast<size_t>(B) * sizeof(int4));
  l.part_o = align_up(l.row_group + static_cast<size_t>(B) * sizeof(int));
  l.part_ml = align_up(l.part_o + part_rows * D * sizeof(float));
  l.tail_o = align_up(l.part_ml + part_rows * sizeof(float2));
  l.tail_ml = align_up(l.tail_o + tail_rows * D * sizeof(float));
  l.total = align_up(l.tail_ml + tail_rows * sizeof(float2));
  return l;
}

template <int D>
kara_status launch_prefix_d(const PrefixArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                            cudaStream_t stream) {
  constexpr size_t smem = PfxSmem<D>::bytes + 1024;
  static std::atomic<int> ready[kMaxDevices];
  const int dev = device_slot();
  if (dev < 0) {
    set_last_error("paged_prefix_attn", "no usable current CUDA device");
    return KARA_ERR_CUDA;
  }
  if (ready[dev].load() == 0) {
    if (cudaFuncSetAttribute(prefix_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
      return check_launch("paged_prefix_attn");
    // the register split draws on what the block is launched with: more would wait forever
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, prefix_attn_kernel<D>) != cudaSuccess)
      return check_launch("paged_prefix_attn");
    if (attr.numRegs * kPfxThreads < 128 * kRegsLow + 2 * kTeamThreads * kRegsHigh) {
      set_last_error("paged_prefix_attn", "the kernel was built with too few registers");
      return KARA_ERR_CUDA;
    }
    ready[dev].store(1);
  }
  launch_pdl(prefix_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
  launch_pdl(prefix_attn_kernel<D>, dim3(static_cast<unsigned>(a.ctas)), dim3(kPfxThreads), smem,
             stream, tk, tv, a);
  return check_launch("paged_prefix_attn");
}

}  // namespace

size_t prefix_workspace_bytes(int B, int Hq, int Hkv, int D) {
  return prefix_layout(B, Hq, Hkv, D).total;
}

kara_status launch_prefix(const PrefixLaunch& L, cudaStream_t stream) {
  const PrefixLayout lay = prefix_layout(L.B, L.Hq, L.Hkv, L.D);
  uint8_t* ws = static_cast<uint8_t*>(L.workspace);
  int sms = 148;
  const int dev = device_slot();
  if (dev >= 0) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  PrefixArgs a;
  a.q = static_cast<const __nv_bfloat16*>(L.q);
  a.block_table = L.block_table;
  a.ctx_len = L.ctx_len;
  a.group_ptr = L.group_ptr;
  a.group_rows = L.group_rows;
  a.prefix_pages = L.prefix_pages;
  a.head = reinterpret_cast<PrefixHead*>(ws + lay.head);
  a.groups = reinterpret_cast<PrefixGroup*>(ws + lay.groups);
  a.rows = reinterpret_cast<int4*>(ws + lay.rows);
  a.row_group = reinterpret_cast<int*>(ws + lay.row_group);
  a.part_o = reinterpret_cast<float*>(ws + lay.part_o);
  a.part_ml = reinterpret_cast<float2*>(ws + lay.part_ml);
  a.status = L.status;
  a.B = L.B;
  a.Hq = L.Hq;
  a.Hkv = L.Hkv;
  a.G = L.Hq / L.Hkv;
  a.max_blocks = L.max_blocks;
  a.num_blocks = L.num_blocks;
  a.num_groups = L.groups;
  a.extra = L.new_slots;
  a.ctas = sms < kMaxCtas ? sms : kMaxCtas;
  a.negate = L.scale < 0.f ? 1 : 0;
  // masked scores are -inf before they are scaled: a scale of 0 becomes the least number, which
  // leaves them -inf and makes 5e-7 of the largest finite score
  a.cs = (a.negate ? -L.scale : L.scale) * 1.4426950408889634f;
  if (a.cs == 0.f) a.cs = std::numeric_limits<float>::denorm_min();
  // the same maps as the streaming kernel's: one page of one KV head, 64 channels per box
  const uint64_t dims[4] = {static_cast<uint64_t>(L.D), static_cast<uint64_t>(L.Hkv), 16,
                            static_cast<uint64_t>(L.num_blocks)};
  const uint64_t strides[3] = {static_cast<uint64_t>(L.D) * 2,
                               static_cast<uint64_t>(L.Hkv) * L.D * 2,
                               static_cast<uint64_t>(16) * L.Hkv * L.D * 2};
  CUtensorMap tk, tv;
  if (!make_bf16_map_4d(&tk, L.k_cache, dims, strides, 16) ||
      !make_bf16_map_4d(&tv, L.v_cache, dims, strides, 16))
    return KARA_ERR_CUDA;
  kara_status st = L.D == 128 ? launch_prefix_d<128>(a, tk, tv, stream)
                              : launch_prefix_d<64>(a, tk, tv, stream);
  if (st != KARA_OK) return st;
  StreamLaunch t;
  t.q = L.q;
  t.k_cache = L.k_cache;
  t.v_cache = L.v_cache;
  t.block_table = L.block_table;
  t.status = L.status;
  t.sel = nullptr;
  t.sel_pages = 0;
  t.line.rows = a.rows;
  t.line.total = &a.head->tail_pages;
  t.line.max_ranges = 0;
  t.line.min_pages = kTailMinPages;
  t.part_o = reinterpret_cast<float*>(ws + lay.tail_o);
  t.part_ml = reinterpret_cast<float2*>(ws + lay.tail_ml);
  t.B = L.B;
  t.Hq = L.Hq;
  t.Hkv = L.Hkv;
  t.D = L.D;
  t.max_blocks = L.max_blocks;
  t.num_blocks = L.num_blocks;
  t.scale = L.scale;
  t.beside = true;
  if ((st = launch_stream(&t, stream)) != KARA_OK) return st;
  JoinLaunch j;
  j.line = t.line;
  j.part_o = t.part_o;
  j.part_ml = t.part_ml;
  j.head = a.head;
  j.groups = a.groups;
  j.row_group = a.row_group;
  j.pre_o = a.part_o;
  j.pre_ml = a.part_ml;
  j.out = L.out;
  j.B = L.B;
  j.Hq = L.Hq;
  j.Hkv = L.Hkv;
  j.D = L.D;
  return launch_join(j, stream);
}

}  // namespace kara
