// Low-rank adapters of many requests beside the shared layer, and their gradients, in
// their simplest form: one block per tile of at most 16 rows of one adapter (or per
// adapter and column block for the weight gradients), fp32 sums in registers.
//
//   forward   h = x A^T (b x r)            y = base + s h B^T
//   backward  dh = s dy B                  dx = base + dh A
//             dA = sum over rows dh^T x    dB = sum over rows s dy^T h
#include <cuda_bf16.h>

#include "twq_adapter.h"

namespace twq {
namespace {

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }
__device__ __forceinline__ uint16_t to_bf(float v) {
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&h);
}

template <bool kCodes>
__device__ __forceinline__ float load_x(const AdapterCall& c, int64_t row, int k) {
  if constexpr (kCodes)
    return static_cast<float>(c.xq8[row * c.m + k]) * c.sx[row * (c.m / 128) + k / 128];
  else
    return bf(c.x[row * c.ldx + k]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}

template <bool kCodes>
__global__ void shrink_kernel(const AdapterCall c, float* hf) {
  if (blockIdx.x >= c.g.tiles[0].x) return;
  const int4 t = c.g.tiles[1 + blockIdx.x];
  const int lane = threadIdx.x & 31;
  for (int p = threadIdx.x >> 5; p < t.z * c.r; p += blockDim.x >> 5) {
    const int64_t row = c.g.order[t.y + p / c.r];
    const int col = p % c.r;
    float v = 0.0f;
    if (t.x >= 0)
      for (int k = lane; k < c.m; k += 32)
        v = fmaf(load_x<kCodes>(c, row, k), bf(c.a[(int64_t(t.x) * c.r + col) * c.m + k]), v);
    v = warp_sum(v);
    if (lane == 0) c.h[row * c.r + col] = to_bf(v);
  }
}

__global__ void expand_kernel(const AdapterCall c) {
  if (blockIdx.x >= c.g.tiles[0].x) return;
  const int4 t = c.g.tiles[1 + blockIdx.x];
  const int j = blockIdx.y * 128 + threadIdx.x;
  for (int i = 0; i < t.z; ++i) {
    const int64_t row = c.g.order[t.y + i];
    float v = 0.0f;
    if (t.x >= 0) {
      for (int k = 0; k < c.r; ++k)
        v = fmaf(bf(c.h[row * c.r + k]), bf(c.bm[(int64_t(t.x) * c.n + j) * c.r + k]), v);
      v *= c.scale[t.x];
    }
    c.y[row * c.n + j] = to_bf((c.base ? bf(c.base[row * c.n + j]) : 0.0f) + v);
  }
}

__global__ void dh_kernel(const AdapterCall c, float* dh) {
  if (blockIdx.x >= c.g.tiles[0].x) return;
  const int4 t = c.g.tiles[1 + blockIdx.x];
  if (t.x < 0) return;
  const int lane = threadIdx.x & 31;
  for (int p = threadIdx.x >> 5; p < t.z * c.r; p += blockDim.x >> 5) {
    const int64_t row = c.g.order[t.y + p / c.r];
    const int col = p % c.r;
    float v = 0.0f;
    for (int k = lane; k < c.n; k += 32)
      v = fmaf(bf(c.dy[row * c.n + k]), bf(c.bm[(int64_t(t.x) * c.n + k) * c.r + col]), v);
    v = warp_sum(v);
    if (lane == 0) dh[row * c.r + col] = v * c.scale[t.x];
  }
}

__global__ void dx_kernel(const AdapterCall c, const float* dh) {
  if (blockIdx.x >= c.g.tiles[0].x) return;
  const int4 t = c.g.tiles[1 + blockIdx.x];
  const int j = blockIdx.y * 128 + threadIdx.x;
  for (int i = 0; i < t.z; ++i) {
    const int64_t row = c.g.order[t.y + i];
    float v = 0.0f;
    if (t.x >= 0)
      for (int k = 0; k < c.r; ++k)
        v = fmaf(dh[row * c.r + k], bf(c.a[(int64_t(t.x) * c.r + k) * c.m + j]), v);
    c.dx[row * c.m + j] = to_bf((c.base ? bf(c.base[row * c.m + j]) : 0.0f) + v);
  }
}

template <bool kCodes>
__global__ void da_kernel(const AdapterCall c, const float* dh) {
  const int j = blockIdx.x * 128 + threadIdx.x, k = blockIdx.y, g = blockIdx.z;
  float v = 0.0f;
  for (int p = c.g.offsets[g]; p < c.g.offsets[g + 1]; ++p) {
    const int64_t row = c.g.order[p];
    v = fmaf(dh[row * c.r + k], load_x<kCodes>(c, row, j), v);
  }
  c.da[(int64_t(g) * c.r + k) * c.m + j] = to_bf(v);
}

__global__ void db_kernel(const AdapterCall c) {
  const int j = blockIdx.x * 128 + threadIdx.x, k = blockIdx.y, g = blockIdx.z;
  float v = 0.0f;
  for (int p = c.g.offsets[g]; p < c.g.offsets[g + 1]; ++p) {
    const int64_t row = c.g.order[p];
    v = fmaf(bf(c.dy[row * c.n + j]), bf(c.h[row * c.r + k]), v);
  }
  c.db[(int64_t(g) * c.n + j) * c.r + k] = to_bf(v * c.scale[g]);
}

}  // namespace

cudaError_t launch_adapter_linear(const AdapterCall& c, cudaStream_t st) {
  if (c.g.b == 0) return cudaSuccess;
  const int cap = row_tiles_cap(c.g.b, c.g.count, 16);
  if (c.xq8)
    shrink_kernel<true><<<cap, 256, 0, st>>>(c, nullptr);
  else
    shrink_kernel<false><<<cap, 256, 0, st>>>(c, nullptr);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  expand_kernel<<<dim3(cap, c.n / 128), 128, 0, st>>>(c);
  return cudaGetLastError();
}

size_t adapter_backward_workspace(int64_t b, int64_t m, int64_t n, int64_t r, int64_t count) {
  (void)m, (void)n, (void)count;
  return static_cast<size_t>(b) * r * 4;
}

cudaError_t launch_adapter_backward(const AdapterCall& c, cudaStream_t st) {
  float* dh = static_cast<float*>(c.workspace);
  cudaError_t e = cudaSuccess;
  if (c.g.b > 0) {
    const int cap = row_tiles_cap(c.g.b, c.g.count, 16);
    dh_kernel<<<cap, 256, 0, st>>>(c, dh);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    dx_kernel<<<dim3(cap, c.m / 128), 128, 0, st>>>(c, dh);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const dim3 ga(c.m / 128, c.r, c.g.count), gb(c.n / 128, c.r, c.g.count);
  if (c.xq8)
    da_kernel<true><<<ga, 128, 0, st>>>(c, dh);
  else
    da_kernel<false><<<ga, 128, 0, st>>>(c, dh);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  db_kernel<<<gb, 128, 0, st>>>(c);
  return cudaGetLastError();
}

}  // namespace twq
