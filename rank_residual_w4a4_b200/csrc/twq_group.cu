// Rows of a batch grouped by adapter: a stable counting sort of the row numbers by id,
// and the lists of row tiles (runs of at most 16 and at most 128 rows of one group) that
// the adapter kernels walk. One block; nothing is read back by the host. Bound by latency: the
// passes over the ids and the barriers between them take 4.5 us for 48 rows and 9.5 us for 16384.
// (Not built: a cluster of blocks for large batches, which could join its counts over distributed
// shared memory.)
#include "twq_adapter.h"

namespace twq {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCountBytes = 160 * 1024;  // shared memory for the per-warp counts

// Exclusive prefix sums over the block of three values per thread.
__device__ __forceinline__ void block_scan3(int (&v)[3], int (&sum)[3], int (*ws)[kWarps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int in[3] = {v[0], v[1], v[2]};
#pragma unroll
  for (int off = 1; off < 32; off <<= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, v[k], off);
      if (lane >= off) v[k] += o;
    }
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < 3; ++k) ws[k][warp] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    int t = ws[k][lane];  // kWarps == 32
    const int mine = t;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, t, off);
      if (lane >= off) t += o;
    }
    sum[k] = __shfl_sync(0xFFFFFFFFu, t, 31);
    v[k] += __shfl_sync(0xFFFFFFFFu, t - mine, warp) - in[k];
  }
}

// Largest key k in [0, n) with first[k] <= t (first is non-decreasing, first[0] == 0 <= t).
__device__ __forceinline__ int find_key(const int* first, int n, int t) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// The keys of rows at, at + 32, ... (-1 from hi on). Their loads go out together: one by one, each
// costs its latency, 16 times over and twice for 16384 rows.
constexpr int kBatch = 16;
__device__ __forceinline__ void load_keys(const int32_t* ids, int at, int hi, int count, int (&key)[kBatch]) {
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int i = at + 32 * u;
    key[u] = i < hi ? __ldg(ids + i) : -1;
  }
#pragma unroll
  for (int u = 0; u < kBatch; ++u)
    if (at + 32 * u < hi && (key[u] < 0 || key[u] >= count)) key[u] = count;
}

// Keys are 0 .. count, key `count` collecting every row whose id is outside [0, count).
// Warp w takes the rows [w * chunk, (w + 1) * chunk) in order: lanes with equal keys
// find each other by a warp match, so a row's rank among its warp's rows of that key
// needs no atomics and the order is the same on every run.
template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    group_rows_kernel(const int32_t* __restrict__ ids, int b, int count, int warps, int chunk,
                      int32_t* order, int32_t* __restrict__ offsets,
                      int4* __restrict__ tiles, int32_t* __restrict__ tiles_before,
                      int cap16) {
  extern __shared__ int smem[];
  __shared__ int ws[3][kWarps];
  const int keys = count + 1;
  int* start = smem;                // rows before the key
  int* first16 = start + keys + 1;  // 16-row tiles before the key
  int* first128 = first16 + keys + 1;
  T* cnt = reinterpret_cast<T*>(first128 + keys + 1);  // warps x keys
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  for (int i = tid; i < warps * keys; i += kThreads) cnt[i] = 0;
  __syncthreads();

  const int lo = min(b, warp * chunk), hi = warp < warps ? min(b, lo + chunk) : lo;
  T* mine = cnt + (warp < warps ? warp : 0) * keys;
  int key[kBatch];
  for (int i = lo; i < hi; i += 32 * kBatch) {
    load_keys(ids, i + lane, hi, count, key);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (i + 32 * u >= hi) break;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, key[u]);
      if (key[u] >= 0 && lane == __ffs(same) - 1) mine[key[u]] = mine[key[u]] + __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();

  // Per key: counts -> rows of the key in earlier warps; totals -> three prefix sums
  // over the keys, each thread taking `per` consecutive ones.
  const int per = (keys + kThreads - 1) / kThreads;
  int v[3] = {0, 0, 0}, sum[3];
  for (int j = 0; j < per; ++j) {
    const int k = tid * per + j;
    if (k >= keys) break;
    int run = 0;
    for (int w = 0; w < warps; ++w) {
      const int c = cnt[w * keys + k];
      cnt[w * keys + k] = static_cast<T>(run);
      run += c;
    }
    start[k] = run;
    v[0] += run;
    v[1] += (run + 15) >> 4;
    v[2] += (run + 127) >> 7;
  }
  block_scan3(v, sum, ws);
  for (int j = 0; j < per; ++j) {
    const int k = tid * per + j;
    if (k >= keys) break;
    const int run = start[k];
    start[k] = v[0];
    first16[k] = v[1];
    first128[k] = v[2];
    tiles_before[k] = v[2];
    offsets[k] = v[0];  // the last key's start is the end of group count - 1
    v[0] += run;
    v[1] += (run + 15) >> 4;
    v[2] += (run + 127) >> 7;
  }
  if (tid == 0) {
    start[keys] = sum[0];
    tiles[0] = make_int4(sum[1], sum[2], 0, 0);
  }
  __syncthreads();

  for (int i = lo; i < hi; i += 32 * kBatch) {
    // a warp's rows are often few enough for the keys to be at hand still
    if (hi - lo > 32 * kBatch) load_keys(ids, i + lane, hi, count, key);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (i + 32 * u >= hi) break;
      const int k = key[u];
      const unsigned same = __match_any_sync(0xFFFFFFFFu, k);
      const int at = k >= 0 ? static_cast<int>(mine[k]) : 0;
      __syncwarp();
      if (k >= 0) {
        order[start[k] + at + __popc(same & ((1u << lane) - 1u))] = i + 32 * u + lane;
        if (lane == __ffs(same) - 1) mine[k] = static_cast<T>(at + __popc(same));
      }
      __syncwarp();
    }
  }

  // Tile lists. The rows of a group ascend, so they follow one another in the batch where the
  // last one is as far from the first as there are rows.
  __syncthreads();
  auto make_tile = [&](int k, int at, int most) {
    const int rows = min(most, start[k + 1] - at);
    const int first = order[at], last = order[at + rows - 1];
    return make_int4(k < count ? k : -1, at, rows, last - first == rows - 1 ? first : -1);
  };
  for (int t = tid; cap16 > 0 && t < sum[1]; t += kThreads) {
    const int k = find_key(first16, keys, t);
    tiles[1 + t] = make_tile(k, start[k] + (t - first16[k]) * 16, 16);
  }
  for (int t = tid; t < sum[2]; t += kThreads) {
    const int k = find_key(first128, keys, t);
    tiles[1 + cap16 + t] = make_tile(k, start[k] + (t - first128[k]) * 128, 128);
  }
}

template <typename T>
cudaError_t launch(const int32_t* ids, int b, const RowGroupsView& g, cudaStream_t st) {
  const int keys = g.count + 1;
  int warps = kCountBytes / (keys * static_cast<int>(sizeof(T)));
  if (warps > kWarps) warps = kWarps;
  int chunk = (b + warps - 1) / warps;
  chunk = (chunk + 31) / 32 * 32;
  const int bytes = 3 * (keys + 1) * 4 + warps * keys * static_cast<int>(sizeof(T));
  const cudaError_t e =
      allow_smem(group_rows_kernel<T>, 3 * (static_cast<int>(kMaxGroups) + 2) * 4 + kCountBytes);
  if (e != cudaSuccess) return e;
  group_rows_kernel<T><<<1, kThreads, bytes, st>>>(
      ids, b, g.count, warps, chunk, g.order, g.offsets, g.tiles, first128_of(g),
      small_tiles_cap(b, g.count));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_group_rows(const int32_t* ids, const RowGroupsView& g, cudaStream_t st) {
  // 16-bit counts where no count can pass 65535: twice the warps for many groups.
  return g.b <= 65535 ? launch<uint16_t>(ids, g.b, g, st) : launch<uint32_t>(ids, g.b, g, st);
}

}  // namespace twq
