// The choice of experts: the k largest logits of each row and their softmax weights.
//
// A warp takes a row and keeps all of it in registers as keys: the bits of a float, mapped so that
// unsigned order is the order of the numbers (a NaN above all, -0 equal to +0, -inf above nothing).
// Each of the k rounds is the lane's own largest key, one reduction of the warp for the key and one
// for the lowest index that has it, so equal logits leave in the order of their indices. A BF16 logit's
// key has 16 bits and leaves room for the index below it: then one reduction does.
//
// Reads 4 (BF16: 2) bytes per logit and writes 8 per choice; what bounds it is latency for a decode
// batch (2.2 us for one row of 128 fp32 logits, mostly launch) and the rounds' instructions for a large
// one (9.4 us for 8192 rows of 256 BF16 logits, 8 choices; issue active 61% of the time).
#include <cuda_bf16.h>

#include "sm100_ptx.cuh"
#include "twq_a16.h"

namespace twq {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kMinusInf = 0x007FFFFFu;  // the key of -inf

__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 + 0 is +0
  if (v != v) return 0xFFFFFFFFu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);  // 0xFFFFFFFF: a NaN
}

// kV: logits per lane.
template <bool kBf16, int kV>
__global__ void __launch_bounds__(kThreads) route_kernel(const __grid_constant__ RouteCall c) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  pdl_wait();
  pdl_launch_dependents();
  if (row >= c.b) return;
  // BF16: the upper half of the key, and 0xFFFF - index.
  constexpr uint32_t kNone = kBf16 ? kMinusInf | 0xFFFFu : kMinusInf;  // no key of a choice is as small
  auto number_of = [](uint32_t k) {  // (~ keeps a negative number's lower half out of the way)
    return kBf16 ? value_of(k & 0x80000000u || k == 0 ? k & 0xFFFF0000u : k | 0xFFFFu) : value_of(k);
  };
  uint32_t key[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int at = i * 32 + lane;
    key[i] = 0;
    if (at < c.count) {
      if constexpr (kBf16) {
        const uint32_t k = key_of(__bfloat162float(static_cast<const __nv_bfloat16*>(c.logits)[row * c.ld + at]));
        key[i] = (k & 0xFFFF0000u) | (0xFFFFu - at);
      } else {
        key[i] = key_of(static_cast<const float*>(c.logits)[row * c.ld + at]);
      }
    }
  }
  float top = 0.0f, sum = 0.0f;
  uint32_t mine = 0;  // the lane-th choice
  int mine_at = -1;
  for (int s = 0; s < c.k; ++s) {
    uint32_t best = key[0], index;
    [[maybe_unused]] int at = 0;
#pragma unroll
    for (int i = 1; i < kV; ++i) {
      if constexpr (kBf16)
        best = max(best, key[i]);
      else if (key[i] > best)
        best = key[i], at = i;
    }
    const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, best);
    if constexpr (kBf16)
      index = 0xFFFFu - (most & 0xFFFFu);
    else
      index = __reduce_min_sync(0xFFFFFFFFu, best == most ? at * 32u + lane : 0xFFFFFFFFu);
    if (s == 0) {
      top = number_of(most);
      if (!c.renormalize) {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const float v = number_of(key[i]);
          if (key[i] > kNone) sum += v == top ? 1.0f : expf(v - top);
        }
      }
    }
    if (most <= kNone) break;
    if (lane == s) mine = most, mine_at = static_cast<int>(index);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      if constexpr (kBf16)
        key[i] = key[i] == most ? 0 : key[i];
      else if (index == i * 32u + lane)
        key[i] = 0;
    }
  }
  const float v = number_of(mine);
  const float e = mine_at < 0 ? 0.0f : v == top ? 1.0f : expf(v - top);
  if (c.renormalize) sum = e;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  if (lane < c.k) {
    c.ids[row * c.k + lane] = mine_at;
    c.weights[row * c.k + lane] = mine_at < 0 ? 0.0f : e / sum;
  }
}

template <bool kBf16, int kV>
cudaError_t launch(const RouteCall& c, cudaStream_t st) {
  constexpr int rows = kThreads / 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((c.b + rows - 1) / rows));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, route_kernel<kBf16, kV>, c);
}

template <bool kBf16>
cudaError_t launch_count(const RouteCall& c, cudaStream_t st) {
  if (c.count <= 32) return launch<kBf16, 1>(c, st);
  if (c.count <= 64) return launch<kBf16, 2>(c, st);
  if (c.count <= 128) return launch<kBf16, 4>(c, st);
  if (c.count <= 256) return launch<kBf16, 8>(c, st);
  if (c.count <= 512) return launch<kBf16, 16>(c, st);
  return launch<kBf16, 32>(c, st);
}

}  // namespace

cudaError_t launch_moe_route(const RouteCall& c, cudaStream_t st) {
  return c.bf16 ? launch_count<true>(c, st) : launch_count<false>(c, st);
}

}  // namespace twq
