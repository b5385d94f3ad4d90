// The adapters' forward pass for small batches (decode steps, a few short prompts): one launch.
// A cluster of 8 blocks takes a tile of at most 16 rows of one adapter. Its 64 warps split the
// reduction over m for h = x A^T, the blocks add their parts over distributed shared memory (in
// rank order, so all hold the same h), and the warps then split n for y = base + s h B^T.
//
// Such a call moves each adapter's A and B once and little else: what bounds it is latency, so
// there is one launch, every warp has its loads of x and A in flight at once, and those of B and
// base for its first columns are issued before h is known. The products go through mma.sync
// m16n8k16: its operands come straight from global memory in 16-byte loads (each weight is used
// by one warp only, so shared memory or tensor memory would only add a step), by giving a lane
// eight consecutive elements of the reduction and both operands the same order.
//
// h takes the place of a BF16 output, and y is made from those same rounded values.
//
// Measured: one row of 4096 x 4096, rank 16, 4.5 us; 48 rows with 20 adapters of 4096 x 14336,
// 7.9 us (15 MB, 1.9 TB/s); 333 rows with 11 of 5120 x 5120, rank 24, 10 us. A warp's groups of 32
// columns of n follow one another, one ahead of the products: two at 4096 columns, seven at 14336.
#include <cuda_bf16.h>

#include <algorithm>

#include "sm100_ptx.cuh"
#include "twq_adapter.h"

namespace twq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRanks = 8;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ float ld_peer(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// base may be y itself: plain accesses, kept in program order.
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void st16(void* p, uint4 v) {
  asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// 8 codes as BF16, which holds them exactly: |c| <= 127 or -128. With 0x43 above it a byte's low
// seven bits make 128 + (c & 127), and its sign bit the 128 or 256 to take off.
__device__ __forceinline__ uint32_t codes2(uint32_t w, uint32_t select) {
  const uint32_t t = __byte_perm(w, 0x43434343u, select);
  uint32_t v = t & 0xFF7FFF7Fu, off = t & 0xFF80FF80u;
  const __nv_bfloat162 d =
      __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), *reinterpret_cast<__nv_bfloat162*>(&off));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint4 codes8(uint2 q) {
  return make_uint4(codes2(q.x, 0x4140), codes2(q.x, 0x4342), codes2(q.y, 0x4140), codes2(q.y, 0x4342));
}

// kR: r rounded up to 16, 32, 64 or 128; ranks from r on are zeros.
template <bool kCodes, int kR>
__global__ void __cluster_dims__(kRanks, 1, 1) __launch_bounds__(kThreads)
    small_kernel(const AdapterCall c) {
  constexpr int kTiles = kR / 8;                        // accumulator tiles of 8 ranks
  constexpr int kUnroll = kR == 16 ? 4 : kR == 32 ? 2 : 1;  // chunks of 32 of m in flight
  constexpr int kSteps = kR == 16 ? 1 : kR / 32;        // loads of a B row per lane (8 or 16 bytes)
  constexpr int kWords = kR == 16 ? 2 : 4;
  extern __shared__ float smem[];                       // kWarps x 16 x kR
  __shared__ float s_part[16 * kR];                     // this block's part of h
  __shared__ __align__(16) uint16_t s_h[16 * (kR + 8)];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x;
  const int number = c.g.tiles[0].x;
  const int4 t = c.g.tiles[1 + blockIdx.y];
  if (static_cast<int>(blockIdx.y) >= number) return;
  const int team = rank * kWarps + warp;  // of kRanks * kWarps warps
  const int q = lane >> 2, t4 = lane & 3;
  if (t.x < 0) {  // rows without adapter: base itself, h = 0
    for (int i = 0; i < t.z; ++i) {
      const int64_t row = c.g.order[t.y + i];
      if (c.base != c.y)
        for (int j = (rank * kThreads + tid) * 8; j < c.n; j += kRanks * kThreads * 8)
          st16(c.y + row * c.n + j, c.base ? ld16(c.base + row * c.n + j) : make_uint4(0, 0, 0, 0));
      if (rank == 0 && tid * 8 < c.r) st16(c.h + row * c.r + tid * 8, make_uint4(0, 0, 0, 0));
    }
    return;
  }
  // rows q and q + 8 of the tile
  const bool ok0 = q < t.z, ok1 = q + 8 < t.z;
  const int64_t row0 = ok0 ? c.g.order[t.y + q] : 0, row1 = ok1 ? c.g.order[t.y + q + 8] : 0;
  const uint4 zero = make_uint4(0, 0, 0, 0);

  // B and base of the warp's first 32 columns, before h is known
  const uint16_t* wb = c.bm + static_cast<int64_t>(t.x) * c.n * c.r;
  uint32_t bw[4][kSteps][kWords];
  uint4 base0 = zero, base1 = zero;
  auto load_b = [&](int group) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // accumulator column 2 t + e of tile j is column 8 t + 2 j + e of the 32
      const uint16_t* src = wb + static_cast<int64_t>(group * 32 + 8 * (q >> 1) + 2 * j + (q & 1)) * c.r;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        if constexpr (kR == 16) {
          const uint2 v = 4 * t4 < c.r ? __ldg(reinterpret_cast<const uint2*>(src + 4 * t4)) : make_uint2(0, 0);
          bw[j][0][0] = v.x, bw[j][0][1] = v.y;
        } else {
          const int at = k * 32 + 8 * t4;
          const uint4 v = at < c.r ? __ldg(reinterpret_cast<const uint4*>(src + at)) : zero;
          bw[j][k][0] = v.x, bw[j][k][1] = v.y, bw[j][k][2] = v.z, bw[j][k][3] = v.w;
        }
      }
    }
  };
  auto load_base = [&](int group) {
    const int col = group * 32 + 8 * t4;
    base0 = c.base && ok0 ? ld16(c.base + row0 * c.n + col) : zero;
    base1 = c.base && ok1 ? ld16(c.base + row1 * c.n + col) : zero;
  };
  constexpr bool kEarly = kR <= 64;  // beyond that the registers go to the accumulators
  const int groups = c.n / 32;
  if (kEarly && team < groups) {
    load_b(team);
    load_base(team);
  }

  // h: chunks of 32 of m, team, team + 64, ...
  float acc[kTiles][4] = {};
  const uint16_t* wa = c.a + static_cast<int64_t>(t.x) * c.r * c.m;
  const int chunks = c.m / 32;
  for (int k0 = team; k0 < chunks; k0 += kRanks * kWarps * kUnroll) {
    uint4 x0[kUnroll], x1[kUnroll], w[kUnroll][kTiles];
    [[maybe_unused]] uint2 q0[kUnroll], q1[kUnroll];
    [[maybe_unused]] float s0[kUnroll], s1[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int chunk = k0 + u * kRanks * kWarps;
      const int at = chunk * 32 + 8 * t4;
      const bool in = chunk < chunks;
      if constexpr (kCodes) {
        q0[u] = in && ok0 ? __ldg(reinterpret_cast<const uint2*>(c.xq8 + row0 * c.m + at)) : make_uint2(0, 0);
        q1[u] = in && ok1 ? __ldg(reinterpret_cast<const uint2*>(c.xq8 + row1 * c.m + at)) : make_uint2(0, 0);
        s0[u] = in && ok0 ? __ldg(c.sx + row0 * (c.m >> 7) + (chunk >> 2)) : 0.0f;
        s1[u] = in && ok1 ? __ldg(c.sx + row1 * (c.m >> 7) + (chunk >> 2)) : 0.0f;
      } else {
        x0[u] = in && ok0 ? __ldg(reinterpret_cast<const uint4*>(c.x + row0 * c.ldx + at)) : zero;
        x1[u] = in && ok1 ? __ldg(reinterpret_cast<const uint4*>(c.x + row1 * c.ldx + at)) : zero;
      }
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
        w[u][j] = in && 8 * j + q < c.r
                      ? __ldg(reinterpret_cast<const uint4*>(wa + static_cast<int64_t>(8 * j + q) * c.m + at))
                      : zero;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if constexpr (kCodes) x0[u] = codes8(q0[u]), x1[u] = codes8(q1[u]);
#pragma unroll
      for (int j = 0; j < kTiles; ++j) {
        // codes: the chunk's sums of code times weight, then each row's scale in fp32
        float part[4] = {};
        float(&d)[4] = kCodes ? part : acc[j];
        mma16816(d, x0[u].x, x1[u].x, x0[u].y, x1[u].y, w[u][j].x, w[u][j].y);
        mma16816(d, x0[u].z, x1[u].z, x0[u].w, x1[u].w, w[u][j].z, w[u][j].w);
        if constexpr (kCodes) {
          acc[j][0] = fmaf(s0[u], part[0], acc[j][0]), acc[j][1] = fmaf(s0[u], part[1], acc[j][1]);
          acc[j][2] = fmaf(s1[u], part[2], acc[j][2]), acc[j][3] = fmaf(s1[u], part[3], acc[j][3]);
        }
      }
    }
  }
  {
    float* p = smem + warp * 16 * kR;
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      *reinterpret_cast<float2*>(p + q * kR + 8 * j + 2 * t4) = make_float2(acc[j][0], acc[j][1]);
      *reinterpret_cast<float2*>(p + (q + 8) * kR + 8 * j + 2 * t4) = make_float2(acc[j][2], acc[j][3]);
    }
  }
  __syncthreads();
  for (int i = tid; i < 16 * kR; i += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += smem[w * 16 * kR + i];
    s_part[i] = v;
  }
  cluster_sync_startup();
  for (int i = tid; i < 16 * kR; i += kThreads) {
    const uint32_t at = smem_u32(s_part + i);
    float o[kRanks], v = 0.0f;
#pragma unroll
    for (int s = 0; s < kRanks; ++s) o[s] = ld_peer(map_peer(at, s));
#pragma unroll
    for (int s = 0; s < kRanks; ++s) v += o[s];
    const int rr = i / kR, col = i % kR;
    // ranks from r on: zero whatever x holds (an infinity times their zero weights is a NaN)
    const uint16_t h = col < c.r ? static_cast<uint16_t>(pack2(v, 0.0f)) : 0;
    s_h[rr * (kR + 8) + col] = h;
    if (rank == 0 && rr < t.z && col < c.r) c.h[static_cast<int64_t>(c.g.order[t.y + rr]) * c.r + col] = h;
  }
  cluster_arrive_release();  // this block has read its peers' parts; waited for at the end
  __syncthreads();

  // y: groups of 32 columns, team, team + 64, ...
  uint32_t ha[kSteps][kWords], hb[kSteps][kWords];  // rows q and q + 8 of h
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const uint32_t* a = reinterpret_cast<const uint32_t*>(s_h + q * (kR + 8)) + (kR == 16 ? 2 * t4 : k * 16 + 4 * t4);
    const uint32_t* b = a + 8 * (kR + 8) / 2;
#pragma unroll
    for (int i = 0; i < kWords; ++i) ha[k][i] = a[i], hb[k][i] = b[i];
  }
  const float f = c.scale[t.x];
  for (int group = team; group < groups; group += kRanks * kWarps) {
    if (!kEarly) {
      load_b(group);
      load_base(group);
    }
    float d[4][4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int i = 0; i < kWords; i += 2)
          mma16816(d[j], ha[k][i], hb[k][i], ha[k][i + 1], hb[k][i + 1], bw[j][k][i], bw[j][k][i + 1]);
    const uint32_t b0[4] = {base0.x, base0.y, base0.z, base0.w}, b1[4] = {base1.x, base1.y, base1.z, base1.w};
    uint32_t o0[4], o1[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o0[j] = pack2(fmaf(f, d[j][0], lo_f(b0[j])), fmaf(f, d[j][1], hi_f(b0[j])));
      o1[j] = pack2(fmaf(f, d[j][2], lo_f(b1[j])), fmaf(f, d[j][3], hi_f(b1[j])));
    }
    const int col = group * 32 + 8 * t4;
    if (kEarly && group + kRanks * kWarps < groups) {
      load_b(group + kRanks * kWarps);
      load_base(group + kRanks * kWarps);
    }
    if (ok0) st16(c.y + row0 * c.n + col, make_uint4(o0[0], o0[1], o0[2], o0[3]));
    if (ok1) st16(c.y + row1 * c.n + col, make_uint4(o1[0], o1[1], o1[2], o1[3]));
  }
  cluster_wait_acquire();  // peers may still be reading this block's part
}

template <bool kCodes, int kR>
cudaError_t launch(const AdapterCall& c, cudaStream_t st) {
  const int smem = kWarps * 16 * kR * 4;
  const cudaError_t e = allow_smem(small_kernel<kCodes, kR>, smem);
  if (e != cudaSuccess) return e;
  small_kernel<kCodes, kR><<<dim3(kRanks, row_tiles_cap(c.g.b, c.g.count, 16)), kThreads, smem, st>>>(c);
  return cudaGetLastError();
}

template <bool kCodes>
cudaError_t launch_rank(const AdapterCall& c, cudaStream_t st) {
  if (c.r <= 16) return launch<kCodes, 16>(c, st);
  if (c.r <= 32) return launch<kCodes, 32>(c, st);
  if (c.r <= 64) return launch<kCodes, 64>(c, st);
  return launch<kCodes, 128>(c, st);
}

}  // namespace

cudaError_t launch_adapter_small(const AdapterCall& c, cudaStream_t st) {
  return c.xq8 ? launch_rank<true>(c, st) : launch_rank<false>(c, st);
}

}  // namespace twq
