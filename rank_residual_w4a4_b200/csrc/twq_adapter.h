// Internal interface of the adapter operators (rows grouped by adapter, low-rank
// adapters beside the layer, their gradients).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/twq.h"

namespace twq {

constexpr int64_t kMaxGroupRows = int64_t(1) << 20;
constexpr int64_t kMaxGroups = 4096;

// Upper bound of the number of tiles of `rows` rows: every group and the rows without
// one can add a partial tile, but a tile holds at least one row.
inline int row_tiles_cap(int64_t b, int64_t count, int rows) {
  const int64_t parts = b < count + 1 ? b : count + 1;
  const int64_t cap = b / rows + parts;
  return static_cast<int>(cap < b ? cap : b);
}

// The forward pass takes the one-launch kernel, on 16-row tiles, for batches up to this many rows
// times rank (from 16 on): its time goes with that, since it reads an adapter again for every 16
// rows. With 4 adapters of 4096 x 4096 it meets the two kernels at about 1000 rows of rank 16
// (16 us), 430 of rank 64 (16 us) and 180 of rank 128 (17 us); of 4096 x 14336 at 620, 260 and 130.
// The rule knows neither m nor n: it changes over at 768, 192 and 96 rows, between or before these.
//
// Twice as many up to rank 16 where the adapters may have 16 rows each or fewer: a row tile of 128
// then holds few rows, but takes the two kernels as long as a full one. 512 rows with 64 adapters of
// 4096 x 4096: 15 us instead of 37, of 4096 x 14336: 33 instead of 70; 1536 rows with 128: 39
// instead of 60, 67 instead of 117. If only 4 of them are used: 23 instead of 25, but 43 instead of
// 34 (which adapters are used is known on the GPU alone).
// (At rank 32: 39 to 39 us, 22 to 22, and 81 to 61 at 14336 x 4096, so not there.)
constexpr int64_t kSmallWork = 12288;
inline bool small_batch(int64_t b, int64_t count, int64_t r) {
  const int64_t work = b * (r > 16 ? r : 16);
  return work <= kSmallWork || (work <= 2 * kSmallWork && r <= 16 && b <= 16 * count);
}
// Room for 16-row tiles: none where no rank makes the batch a small one.
inline int small_tiles_cap(int64_t b, int64_t count) {
  return small_batch(b, count, 1) ? row_tiles_cap(b, count, 16) : 0;
}

// tiles: {number of 16-row tiles, number of 128-row tiles, 0, 0}, then room for
// small_tiles_cap(b, count) entries of the first list and row_tiles_cap(b, count, 128) of the second;
// an entry is {group or -1, first position in order, rows, first row where the rows follow one
// another in the batch, else -1}. After the entries: for each group, then for the rows without
// one, the 128-row tiles before it (count + 1 integers).
struct RowGroupsView {
  int b, count;
  int32_t* order;
  int32_t* offsets;
  int4* tiles;
};

inline int32_t* first128_of(const RowGroupsView& g) {
  return reinterpret_cast<int32_t*>(g.tiles + 1 + small_tiles_cap(g.b, g.count) +
                                    row_tiles_cap(g.b, g.count, 128));
}

cudaError_t launch_group_rows(const int32_t* ids, const RowGroupsView& g, cudaStream_t st);

// Allows `kernel` `smem` bytes of dynamic shared memory (its largest use), once per device and again
// after twq_release_cache.
cudaError_t allow_smem(const void* kernel, int smem);
template <typename Kernel>
cudaError_t allow_smem(Kernel* kernel, int smem) {
  return allow_smem(reinterpret_cast<const void*>(kernel), smem);
}
// twq_release_cache: forget for which kernels that was done (a reset of the device undoes it).
void release_adapter_cache();

struct AdapterCall {
  RowGroupsView g;
  int m, n, r;
  const uint16_t* a;    // count x r x m
  const uint16_t* bm;   // count x n x r
  const float* scale;   // count
  const uint16_t* x;    // BF16 X (row stride ldx), or null with codes
  int64_t ldx;
  const int8_t* xq8;    // 8-bit codes, b x m, or null
  const float* sx;      // their scales, b x m/128
  const uint16_t* base; // b x n (forward) or b x m (backward), or null
  uint16_t* h;          // b x r: output of the forward pass, input of the backward pass
  uint16_t* y;          // forward: b x n
  const uint16_t* dy;   // backward: b x n
  uint16_t* dx;         // b x m
  uint16_t* da;         // count x r x m
  uint16_t* db;         // count x n x r
  void* workspace;
  uint64_t wait_ns;     // limit of the kernels' waits
  int stall;            // self-test: a loading warp stops early, so that the waits on it run out
};
constexpr uint64_t kAdapterWaitNs = 2000000000ull;

cudaError_t launch_adapter_linear(const AdapterCall& c, cudaStream_t st);
// The forward pass for small batches (16-row tiles, one launch).
cudaError_t launch_adapter_small(const AdapterCall& c, cudaStream_t st);
cudaError_t launch_adapter_backward(const AdapterCall& c, cudaStream_t st);
cudaError_t read_and_clear_adapter_status(int* code);
size_t adapter_backward_workspace(int64_t b, int64_t m, int64_t n, int64_t r, int64_t count);

}  // namespace twq
