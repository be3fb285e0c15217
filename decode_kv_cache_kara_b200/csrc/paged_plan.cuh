// What the kernels of one block-sparse or shared-prefix attention call hand to each other.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kara.h"

namespace kara {

// The pages that the streaming kernel reads form one line per KV head, row after row. Row i of
// the line: (cache row or -1, its first page, its slots, where it starts on the line).
// The line is cut into R equal ranges, one per warp and KV head; a range leaves one partial
// (m, l, o) per row that it touches, in slot i + range: along the line either number grows from
// one partial to the next, so slots are never shared.
struct StreamLine {
  const int4* rows;      // [B]
  const int* total;      // pages on the line
  int max_ranges;        // ranges that the launch can run at once
  int min_pages;         // pages that are worth a range
};
__device__ __forceinline__ int stream_ranges(const StreamLine& s, int total) {
  const int most = total / s.min_pages;
  return total == 0 ? 0 : most < 1 ? 1 : most < s.max_ranges ? most : s.max_ranges;
}
// n / d for n >= 0, d > 0: the 64-bit division only where one of them needs it.
__host__ __device__ __forceinline__ long long divide(long long n, long long d) {
  return ((n | d) >> 32) == 0
             ? static_cast<long long>(static_cast<uint32_t>(n) / static_cast<uint32_t>(d))
             : n / d;
}
// A line of `total` units cut into `parts` equal parts: the first unit of part r, and the part that
// holds unit u.
__host__ __device__ __forceinline__ long long part_start(long long r, int parts, long long total) {
  return divide(r * total, parts);
}
__host__ __device__ __forceinline__ int part_of(long long u, int parts, long long total) {
  return static_cast<int>(divide((u + 1) * parts - 1, total));
}
// First page of range r of R on a line of `total` pages, and the range that holds page p.
__device__ __forceinline__ int range_start(int r, int R, int total) {
  return static_cast<int>(part_start(r, R, total));
}
__device__ __forceinline__ int range_of(int p, int R, int total) { return part_of(p, R, total); }

// Shared prefixes: the work of all items (group, query tile, KV head) is one line of key tiles,
// cut into equal parts, one per block.
constexpr int kItemRows = 256;          // query rows per item, at most
constexpr int kItemCost = 3;            // an item's start and end, in key tiles
struct PrefixHead {
  long long total;       // work of all items, in key tiles
  int ctas;              // blocks with prefix work
  int tail_pages;        // the streaming kernel's line
};
struct PrefixGroup {
  long long flat;        // work of the groups before
  int first, rows;       // list positions [first, first + rows)
  int ktiles;            // key tiles per item (0: no shared part)
  int pages;             // prefix pages
  int row0;              // cache row whose table names the prefix pages
  int item_rows;         // query rows per item (fewer in the last)
};

struct StreamLaunch {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_table;
  int32_t* status;
  const int32_t* sel;    // [B, Hkv, sel_pages]: the line's pages are entries of these lists
  int sel_pages;
  StreamLine line;
  float* part_o;         // [B + max_ranges, Hq, D]
  float2* part_ml;       // [B + max_ranges, Hq]
  int B, Hq, Hkv, D, max_blocks, num_blocks;
  float scale;
  // runs beside the kernel launched before it: the line was written before that one, and this
  // one waits for it at its end
  bool beside;
};
int stream_max_ranges(int hkv);          // bound that sizes workspaces
kara_status launch_stream(StreamLaunch* L, cudaStream_t stream);   // sets line.max_ranges

struct JoinLaunch {
  StreamLine line;
  const float* part_o;
  const float2* part_ml;
  // the prefix partials, or null: [B Hq + kItemRows blocks] rows
  const PrefixHead* head;
  const PrefixGroup* groups;
  const int* row_group;
  const float* pre_o;
  const float2* pre_ml;
  void* out;
  int B, Hq, Hkv, D;
};
kara_status launch_join(const JoinLaunch& L, cudaStream_t stream);

}  // namespace kara
