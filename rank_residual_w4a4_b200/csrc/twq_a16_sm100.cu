// Products of few rows of BF16 activations with packed 4-bit weights: the layer itself for up to
// 64 tokens, and the gated products of the experts that a router chose.
//
// A group's sum over its 128 codes is taken exactly as in the quantized layer, only that the other
// operand is BF16: codes are small integers, which BF16 holds, so mma.sync m16n8k16 multiplies them
// exactly and sums in fp32, and the group's fp32 scale multiplies that sum once.
//
// Few rows make this a stream of weights: what bounds it is HBM, or latency where the weights are
// few. So every warp has a ring of its own in shared memory that it fills with cp.async, no
// thread waits for another one's copies, and the reduction is split as far as it takes to have all
// SMs load: over warps, and over the blocks of a cluster, which add up over distributed shared
// memory in a fixed order. The weights are the M side of the products, 32 columns of them to a
// warp, rows of activations the N side, 8 to a tile.
//
// A unit of a warp's work is 32 weight columns x one group of 128: 16 bytes (32 codes) per lane and
// column, as they lie in memory. The order in which a lane's 32 codes go through the products is
// free as long as the activations follow it: codes i and i + 4 of a word become one BF16 pair by one
// logic operation (0x4300 | (code ^ 8) is 136 + code) and one exact subtraction. The low-rank
// factor L2 comes last, as units of 32 columns x 32 ranks.
#include <cuda_bf16.h>

#include <algorithm>

#include "sm100_ptx.cuh"
#include "twq_a16.h"
#include "twq_adapter.h"

namespace twq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 4;
constexpr int kRows = 32;                 // weight columns of a unit (rows of the packed codes)
constexpr int kStageBytes = kRows * 64 + kRows * 4;
constexpr int kYStride = 40;              // floats between the rows of a warp's sums
constexpr int kSms = 148;

enum Mode : int {
  kModeH = 0,    // h = bf16(x D(L1))
  kModeAct = 1,  // a = silu(g) u, in two BF16 terms
  kModeY = 2,    // y = base + sum of weight * (x D(R) + h L2)
};

struct A16Args {
  const uint8_t* q;     // codes: n x K/2 per expert
  const float* s;       // scales: K/128 x n per expert
  const uint16_t* l2t;  // n x r per expert (kModeH: none)
  int64_t q_expert, s_expert, l2_expert;  // elements from one expert to the next
  int K, n, r;          // r: ranks of l2t read here
  int f;                // kModeAct: gate columns (n = 2 f)
  const uint16_t* x;    // token rows (row stride ldx), or the pairs' activations
  const uint16_t* x_lo; // kParts == 2: the activations' second terms
  int64_t ldx;
  const uint16_t* h;    // low-rank input, tokens or pairs x r
  const int32_t* ids;   // b x k
  const float* weights; // b x k
  int b, k, count;
  const uint16_t* base; // kModeY
  uint16_t* out;
  uint16_t* out_lo;     // kModeAct
  int tiles;            // column tiles of a chunk
  int split;            // blocks of a cluster
  bool ids_ready, x_ready;  // complete before this kernel starts, whatever it waits for
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Activations may come from the kernel that this one overlaps: plain loads, kept in order.
__device__ __forceinline__ uint4 ld16(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld4(const void* p) {
  uint32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float lds_f(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_peer(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// 16 bytes into shared memory; zeros where `in` is false (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Codes i and i + 4 of a word (shifted right by 4 i) as a BF16 pair.
__device__ __forceinline__ uint32_t codes2(uint32_t w) {
  uint32_t t;
  asm("lop3.b32 %0, %1, 0x000F000F, 0x43084308, 0x6A;" : "=r"(t) : "r"(w));  // (w & mask) ^ bits: 136 + code
  const uint32_t off = 0x43084308u;
  const __nv_bfloat162 d =
      __hsub2(*reinterpret_cast<__nv_bfloat162*>(&t), *reinterpret_cast<const __nv_bfloat162*>(&off));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// What of a block's shared memory is where, in bytes. pairs: b x k.
struct Layout {
  int ring, sums, part, chunks, order, cnt, total;
};
template <int NT, int kMode, int kParts, bool kRouted>
__host__ __device__ inline Layout layout(int b, int k, int count, int split) {
  constexpr int cap = 8 * NT / kParts;
  const int pairs = kRouted ? b * k : b;
  const int rows = kMode == kModeY ? b : cap;
  const int buffers = kMode == kModeY ? 1 : 2;
  const int groups = pairs < count ? pairs : count;
  const int chunks = kRouted ? (groups + pairs / cap < pairs ? groups + pairs / cap : pairs) : 0;
  Layout l;
  l.ring = 0;
  l.sums = l.ring + kWarps * kStages * kStageBytes;
  l.part = l.sums + buffers * kWarps * rows * kYStride * 4;
  l.chunks = l.part + (split > 1 ? buffers * rows * kRows * 4 : 0);
  l.order = l.chunks + chunks * 8;
  l.cnt = l.order + (kRouted ? 2 * ((pairs * 2 + 7) / 8 * 8) : 0);
  l.total = l.cnt + (kRouted ? count * 4 : 0);
  l.total = (l.total + 15) / 16 * 16;
  return l;
}

template <int NT, int kMode, int kParts, bool kRouted>
__global__ void __launch_bounds__(kThreads, NT <= 2 ? 2 : 1) a16_kernel(const __grid_constant__ A16Args a) {
  constexpr int kCap = 8 * NT / kParts;  // rows of activations in a chunk
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int s_chunks, s_twice;
  const Layout lay = layout<NT, kMode, kParts, kRouted>(a.b, a.k, a.count, a.split);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % a.split, cluster = blockIdx.x / a.split;
  const int clusters = gridDim.x / a.split;
  uint2* s_chunk = reinterpret_cast<uint2*>(smem + lay.chunks);
  uint16_t* s_order = reinterpret_cast<uint16_t*>(smem + lay.order);
  const int pairs = kRouted ? a.b * a.k : a.b;

  bool waited = false;
  auto wait_all = [&] {
    if (!waited) pdl_wait();
    waited = true;
  };
  if (!a.ids_ready) {
    wait_all();
    pdl_launch_dependents();
  }

  // Chunks of at most kCap rows that share an expert, experts ascending, rows of an expert in the
  // order of their pairs: {expert, first place in s_order | rows << 16}.
  if constexpr (kRouted) {
    int* s_cnt = reinterpret_cast<int*>(smem + lay.cnt);
    uint16_t* s_rank = s_order + (pairs * 2 + 7) / 8 * 4;
    for (int i = tid; i < a.count; i += kThreads) s_cnt[i] = 0;
    if (tid == 0) s_twice = 0;
    __syncthreads();
    if (warp == 0) {
      for (int p0 = 0; p0 < pairs; p0 += 32) {
        const int p = p0 + lane;
        int id = p < pairs ? static_cast<int>(ld4(a.ids + p)) : -1;
        if (id < 0 || id >= a.count) id = -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
        const int at = id >= 0 ? s_cnt[id] : 0;
        __syncwarp();
        if (id >= 0) {
          s_rank[p] = static_cast<uint16_t>(at + __popc(same & ((1u << lane) - 1u)));
          if (lane == __ffs(same) - 1) s_cnt[id] = at + __popc(same);
        }
        __syncwarp();
      }
      int rows = 0, chunks = 0;
      for (int e0 = 0; e0 < a.count; e0 += 32) {
        const int e = e0 + lane;
        const int c = e < a.count ? s_cnt[e] : 0;
        const int n = (c + kCap - 1) / kCap;
        int rs = c, cs = n;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const int r2 = __shfl_up_sync(0xFFFFFFFFu, rs, d), c2 = __shfl_up_sync(0xFFFFFFFFu, cs, d);
          if (lane >= d) rs += r2, cs += c2;
        }
        const int first = rows + rs - c;
        if (e < a.count) s_cnt[e] = first;
        for (int i = 0; i < n; ++i)
          s_chunk[chunks + cs - n + i] =
              make_uint2(e, (first + i * kCap) | (min(kCap, c - i * kCap) << 16));
        rows += __shfl_sync(0xFFFFFFFFu, rs, 31);
        chunks += __shfl_sync(0xFFFFFFFFu, cs, 31);
      }
      if (lane == 0) s_chunks = chunks;
    }
    __syncthreads();
    for (int p = tid; p < pairs; p += kThreads) {
      const int id = static_cast<int>(ld4(a.ids + p));
      if (id < 0 || id >= a.count) continue;
      s_order[s_cnt[id] + s_rank[p]] = static_cast<uint16_t>(p);
      // an expert twice among one token's
      for (int o = p - p % a.k; o < p; ++o)
        if (static_cast<int>(ld4(a.ids + o)) == id) s_twice = 1;
    }
    __syncthreads();
  }
  const int chunks = kRouted ? s_chunks : (a.b + kCap - 1) / kCap;
  auto chunk_expert = [&](int c) { return kRouted ? static_cast<int>(s_chunk[c].x) : 0; };
  auto chunk_first = [&](int c) { return kRouted ? static_cast<int>(s_chunk[c].y & 0xFFFFu) : c * kCap; };
  auto chunk_rows = [&](int c) {
    return kRouted ? static_cast<int>(s_chunk[c].y >> 16) : min(kCap, a.b - c * kCap);
  };

  // The warp's share of the units. kModeY: of all chunks' units of one column tile; else of every
  // job's, a job being a chunk and a column tile.
  const int groups = a.K >> 7, per = groups + (a.r + 31) / 32;
  const int team = rank * kWarps + warp, teams = a.split * kWarps;
  const int total = kMode == kModeY ? chunks * per : per;
  const int lo = static_cast<int>(static_cast<int64_t>(total) * team / teams);
  const int hi = static_cast<int>(static_cast<int64_t>(total) * (team + 1) / teams);
  const int jobs = kMode == kModeY ? a.tiles : chunks * a.tiles;

  // Column (row of the codes) that lane quad g loads for 8-row part i of tile `tile`, or -1.
  const uint32_t ring = smem_u32(smem + lay.ring) + warp * kStages * kStageBytes;
  const int64_t half = a.K >> 1;
  auto column = [&](int tile, int i) {
    if constexpr (kMode == kModeAct) return (i >> 1) * a.f + tile * 16 + (i & 1) * 8 + g;
    const int c = tile * kRows + i * 8 + g;
    return c < a.n ? c : -1;
  };

  // Copies, kStages - 1 units ahead.
  struct {
    int job, chunk, tile, u, left;
  } p = {cluster, 0, 0, 0, 0};
  auto start_job = [&] {
    p.left = p.job < jobs ? hi - lo : 0;
    if (p.left <= 0) return;
    if constexpr (kMode == kModeY) {
      p.tile = p.job, p.chunk = lo / per, p.u = lo % per;
    } else {
      p.chunk = p.job / a.tiles, p.tile = p.job - p.chunk * a.tiles, p.u = lo;
    }
  };
  start_job();
  auto request = [&](int stage) {
    if (p.left > 0) {
      const uint32_t dst = ring + stage * kStageBytes;
      const int64_t e = chunk_expert(p.chunk);
      if (p.u < groups) {
        const uint8_t* q = a.q + e * a.q_expert + p.u * 64 + t * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = column(p.tile, i);
          copy16(dst + i * 512 + lane * 16, c >= 0 ? q + c * half : q, c >= 0);
        }
        if (lane < 8) {  // four scales each
          int c = kMode == kModeAct ? (lane >> 2) * a.f + p.tile * 16 + (lane & 3) * 4 : p.tile * kRows + lane * 4;
          const bool in = c < a.n;
          if (!in) c = 0;
          copy16(dst + kRows * 64 + lane * 16, a.s + e * a.s_expert + static_cast<int64_t>(p.u) * a.n + c, in);
        }
      } else {
        const int at = (p.u - groups) * 32 + t * 8;
        const uint16_t* l2 = a.l2t + e * a.l2_expert;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = column(p.tile, i);
          const bool in = c >= 0 && at < a.r;
          copy16(dst + i * 512 + lane * 16, in ? l2 + static_cast<int64_t>(c) * a.r + at : l2, in);
        }
      }
      --p.left;
      if (++p.u == per) p.u = 0, ++p.chunk;
      if (p.left == 0) {
        p.job += clusters;
        start_job();
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) request(i);

  if (!a.x_ready) wait_all();
  if (a.ids_ready) pdl_launch_dependents();

  int stage = 0;
  float* const sums = reinterpret_cast<float*>(smem + lay.sums);
  constexpr int kBuffers = kMode == kModeY ? 1 : 2;
  const int srows = kMode == kModeY ? a.b : kCap;
  float* const part = reinterpret_cast<float*>(smem + lay.part);
  int buffer = 0;
  for (int job = cluster; job < jobs; job += clusters) {
    float* const mine = sums + (buffer * kWarps + warp) * srows * kYStride;
    int chunk, u;
    const int tile = kMode == kModeY ? job : job % a.tiles;
    if constexpr (kMode == kModeY) {
      chunk = lo / per, u = lo % per;
      for (int i = lane; i < srows * kYStride; i += 32) mine[i] = 0.0f;
      __syncwarp();
    } else {
      chunk = job / a.tiles, u = lo;
    }
    float acc[2][NT][4];
    const uint16_t* row[NT];
    auto enter_chunk = [&] {
      const int first = chunk_first(chunk), rows = chunk_rows(chunk);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int col = nt * 8 + g, i = kParts == 2 ? col >> 1 : col;
        row[nt] = nullptr;
        if (i < rows) {
          const int pr = kRouted ? s_order[first + i] : first + i;
          const int64_t at = kRouted && kParts == 1 ? pr / a.k : pr;
          row[nt] = (kParts == 2 && (col & 1) ? a.x_lo : a.x) + at * a.ldx;
        }
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i2][nt][j] = 0.0f;
      }
    };
    // Adds (kModeY) or stores the chunk's sums to the warp's own rows.
    auto leave_chunk = [&] {
      const int first = chunk_first(chunk), rows = chunk_rows(chunk);
      auto put = [&](int i, float v0, float v1, float v2, float v3) {
        if (i >= rows) return;
        int at = i;
        float f = 1.0f;
        if constexpr (kMode == kModeY) {
          const int pr = kRouted ? s_order[first + i] : first + i;
          at = kRouted ? pr / a.k : pr;
          if (kRouted) f = a.weights[pr];
        }
        float* y = mine + at * kYStride + g;
        const float v[4] = {v0, v1, v2, v3};
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j * 8] = kMode == kModeY ? fmaf(f, v[j], y[j * 8]) : v[j];
      };
      auto put_all = [&] {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (kParts == 2) {
            put(nt * 4 + t, acc[0][nt][0] + acc[0][nt][1], acc[0][nt][2] + acc[0][nt][3],
                acc[1][nt][0] + acc[1][nt][1], acc[1][nt][2] + acc[1][nt][3]);
          } else {
            put(nt * 8 + 2 * t, acc[0][nt][0], acc[0][nt][2], acc[1][nt][0], acc[1][nt][2]);
            put(nt * 8 + 2 * t + 1, acc[0][nt][1], acc[0][nt][3], acc[1][nt][1], acc[1][nt][3]);
          }
        }
      };
      if (kMode == kModeY && kRouted && s_twice) {  // two pairs of a chunk may be one token's
        for (int o = 0; o < 4; ++o) {
          if (t == o) put_all();
          __syncwarp();
        }
      } else {
        put_all();
        __syncwarp();
      }
    };
    if (lo < hi) enter_chunk();
    for (int v = lo; v < hi; ++v) {
      copy_wait<kStages - 2>();
      __syncwarp();
      request(stage == 0 ? kStages - 1 : stage - 1);
      const uint32_t src = ring + stage * kStageBytes;
      stage = stage == kStages - 1 ? 0 : stage + 1;
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = lds16(src + i * 512 + lane * 16);
      if (u < groups) {
        float s[4], d[2][NT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = lds_f(src + kRows * 64 + (i * 8 + g) * 4);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) d[i][nt][j] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 x[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            x[nt] = row[nt] ? ld16(row[nt] + u * 128 + t * 32 + j * 8) : make_uint4(0, 0, 0, 0);
          uint32_t c[2][2][4];  // tile, code i & 3, {rows g: i, i + 4 ...}
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 w0 = w[2 * i], w1 = w[2 * i + 1];
            const uint32_t a0 = j == 0 ? w0.x : j == 1 ? w0.y : j == 2 ? w0.z : w0.w;
            const uint32_t a1 = j == 0 ? w1.x : j == 1 ? w1.y : j == 2 ? w1.z : w1.w;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              c[i][k][0] = codes2(a0 >> (8 * k)), c[i][k][1] = codes2(a1 >> (8 * k));
              c[i][k][2] = codes2(a0 >> (8 * k + 4)), c[i][k][3] = codes2(a1 >> (8 * k + 4));
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t b0 = __byte_perm(x[nt].x, x[nt].z, 0x5410), b1 = __byte_perm(x[nt].x, x[nt].z, 0x7632);
            const uint32_t b2 = __byte_perm(x[nt].y, x[nt].w, 0x5410), b3 = __byte_perm(x[nt].y, x[nt].w, 0x7632);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              mma16816(d[i][nt], c[i][0][0], c[i][0][1], c[i][0][2], c[i][0][3], b0, b1);
              mma16816(d[i][nt], c[i][1][0], c[i][1][1], c[i][1][2], c[i][1][3], b2, b3);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            acc[i][nt][0] = fmaf(s[2 * i], d[i][nt][0], acc[i][nt][0]);
            acc[i][nt][1] = fmaf(s[2 * i], d[i][nt][1], acc[i][nt][1]);
            acc[i][nt][2] = fmaf(s[2 * i + 1], d[i][nt][2], acc[i][nt][2]);
            acc[i][nt][3] = fmaf(s[2 * i + 1], d[i][nt][3], acc[i][nt][3]);
          }
      } else {
        wait_all();
        const int at = (u - groups) * 32 + t * 8, first = chunk_first(chunk), rows = chunk_rows(chunk);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int col = nt * 8 + g, i = kParts == 2 ? col >> 1 : col;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (i < rows && !(kParts == 2 && (col & 1)) && at < a.r) {
            const int64_t pr = kRouted ? s_order[first + i] : first + i;
            x = ld16(a.h + pr * a.r + at);
          }
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2) {
            mma16816(acc[i2][nt], w[2 * i2].x, w[2 * i2 + 1].x, w[2 * i2].y, w[2 * i2 + 1].y, x.x, x.y);
            mma16816(acc[i2][nt], w[2 * i2].z, w[2 * i2 + 1].z, w[2 * i2].w, w[2 * i2 + 1].w, x.z, x.w);
          }
        }
      }
      if (++u == per || v + 1 == hi) {
        leave_chunk();
        u = 0, ++chunk;
        if (v + 1 < hi) enter_chunk();
      }
    }
    if constexpr (kMode != kModeY) {
      if (lo >= hi)
        for (int i = lane; i < srows * kYStride; i += 32) mine[i] = 0.0f;
    }
    __syncthreads();

    // The block's sum of its warps, then the cluster's of its blocks, each in order.
    const int job_chunk = kMode == kModeY ? 0 : job / a.tiles;
    const int first = kMode == kModeY ? 0 : chunk_first(job_chunk);
    const int rows = kMode == kModeY ? a.b : chunk_rows(job_chunk);
    const float* all = sums + buffer * kWarps * srows * kYStride;
    float* const own = part + buffer * srows * kRows;
    auto block_sum = [&](int r2, int c) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += all[(w * srows + r2) * kYStride + c];
      return v;
    };
    if (a.split > 1) {
      for (int i = tid; i < rows * kRows; i += kThreads) own[i] = block_sum(i >> 5, i & 31);
      cluster_sync_startup();
    }
    auto sum = [&](int r2, int c) {
      if (a.split == 1) return block_sum(r2, c);
      const uint32_t at = smem_u32(own + r2 * kRows + c);
      float v = 0.0f;
      for (int s = 0; s < a.split; ++s) v += ld_peer(map_peer(at, s));
      return v;
    };
    // Two neighbouring values per thread; the blocks of a cluster share the pairs out.
    constexpr int kWide = kMode == kModeAct ? 8 : 16;
    for (int i = rank * kThreads + tid; i < rows * kWide; i += a.split * kThreads) {
      const int r2 = i / kWide, c = 2 * (i % kWide);
      if constexpr (kMode == kModeAct) {
        const int64_t at = static_cast<int64_t>(kRouted ? s_order[first + r2] : first + r2) * a.f + tile * 16 + c;
        float v[2], hi2[2], lo2[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float gate = sum(r2, c + e), up = sum(r2, 16 + c + e);
          v[e] = gate / (1.0f + expf(-gate)) * up;
          hi2[e] = __bfloat162float(__float2bfloat16_rn(v[e]));
          lo2[e] = isfinite(hi2[e]) ? v[e] - hi2[e] : 0.0f;
        }
        *reinterpret_cast<uint32_t*>(a.out + at) = pack2(hi2[0], hi2[1]);
        *reinterpret_cast<uint32_t*>(a.out_lo + at) = pack2(lo2[0], lo2[1]);
      } else {
        const int col = tile * kRows + c;
        if (col >= a.n) continue;
        float v0 = sum(r2, c), v1 = sum(r2, c + 1);
        const int64_t pr = kMode == kModeY ? r2 : kRouted ? s_order[first + r2] : first + r2;
        const int64_t at = pr * a.n + col;
        if (kMode == kModeY && a.base) {
          const uint32_t bv = ld4(a.base + at);
          v0 += lo_f(bv), v1 += hi_f(bv);
        }
        *reinterpret_cast<uint32_t*>(a.out + at) = pack2(v0, v1);
      }
    }
    if (kBuffers == 2) buffer ^= 1;
  }
  wait_all();  // this grid completes only after the one in front
  if (a.split > 1) cluster_sync_startup();  // peers may still be reading this block's sums
}

template <int NT, int kMode, int kParts, bool kRouted>
cudaError_t launch(A16Args a, int64_t jobs, cudaStream_t st) {
  auto kernel = a16_kernel<NT, kMode, kParts, kRouted>;
  // Blocks of a cluster: as many as it takes for two blocks on every SM, while each of their warps
  // has a unit still.
  const int64_t units = a.K / 128 + (a.r + 31) / 32;
  a.split = 1;
  while (a.split < 8 && jobs * a.split * 2 <= 2 * kSms && units >= 2 * a.split * kWarps) a.split *= 2;
  const Layout l = layout<NT, kMode, kParts, kRouted>(a.b, a.k, a.count, a.split);
  const cudaError_t e = allow_smem(kernel, 227 * 1024 - 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int64_t most = kMode == kModeY ? jobs : std::min<int64_t>(jobs, 4 * kSms / a.split);
  cfg.gridDim = dim3(static_cast<unsigned>(most * a.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = l.total;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = a.split;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Rows of activations that a chunk has to hold: 8, 16 or 32.
template <int kMode, int kParts, bool kRouted>
cudaError_t launch_rows(const A16Args& a, int rows, int64_t jobs_of_pairs, cudaStream_t st) {
  const int64_t tiles = a.tiles;
  auto jobs = [&](int cap) {
    if (kMode == kModeY) return tiles;
    const int64_t pairs = jobs_of_pairs;
    const int64_t groups = kRouted ? std::min<int64_t>(pairs, a.count) : 1;
    return tiles * (kRouted ? std::min(pairs, groups + pairs / cap) : (pairs + cap - 1) / cap);
  };
  if (rows * kParts <= 8) return launch<1, kMode, kParts, kRouted>(a, jobs(8 / kParts), st);
  if (rows * kParts <= 16) return launch<2, kMode, kParts, kRouted>(a, jobs(16 / kParts), st);
  return launch<4, kMode, kParts, kRouted>(a, jobs(32 / kParts), st);
}

A16Args product(const uint8_t* q, const float* s, const uint16_t* l2t, int64_t K, int64_t n, int64_t r) {
  A16Args a = {};
  a.q = q, a.s = s, a.l2t = l2t;
  a.K = static_cast<int>(K), a.n = static_cast<int>(n), a.r = static_cast<int>(r);
  a.q_expert = n * (K / 2), a.s_expert = n * (K / 128), a.l2_expert = n * r;
  a.tiles = static_cast<int>((n + kRows - 1) / kRows);
  a.k = 1, a.count = 1;
  return a;
}

size_t up16(size_t v) { return (v + 15) & ~size_t(15); }

}  // namespace

cudaError_t launch_a16_linear(const A16LinearCall& c, cudaStream_t st) {
  const twq_weights& w = *c.w;
  if (w.r > 0) {
    A16Args a = product(w.l1q, w.sl1, nullptr, w.m, w.r, 0);
    a.x = c.x, a.ldx = c.ldx, a.b = c.b, a.out = c.h;
    a.ids_ready = true;
    const cudaError_t e = launch_rows<kModeH, 1, false>(a, c.b, c.b, st);
    if (e != cudaSuccess) return e;
  }
  A16Args a = product(w.rq, w.sr, w.l2t, w.m, w.n, w.r);
  a.x = c.x, a.ldx = c.ldx, a.b = c.b, a.h = c.h, a.out = c.y;
  a.ids_ready = true, a.x_ready = w.r > 0;
  return launch_rows<kModeY, 1, false>(a, c.b, c.b, st);
}

size_t moe_workspace(int64_t pairs, const twq_experts* e) {
  return 2 * up16(2 * pairs * e->down.m) + up16(2 * pairs * e->up.r) + up16(2 * pairs * e->down.r);
}

cudaError_t launch_moe_experts(const MoeCall& c, cudaStream_t st) {
  const twq_weights &u = c.e->up, &d = c.e->down;
  const int64_t pairs = int64_t(c.b) * c.k, f = d.m;
  uint8_t* ws = static_cast<uint8_t*>(c.workspace);
  uint16_t* act = reinterpret_cast<uint16_t*>(ws);
  uint16_t* act_lo = reinterpret_cast<uint16_t*>(ws + up16(2 * pairs * f));
  uint16_t* h1 = reinterpret_cast<uint16_t*>(ws + 2 * up16(2 * pairs * f));
  uint16_t* h2 = reinterpret_cast<uint16_t*>(ws + 2 * up16(2 * pairs * f) + up16(2 * pairs * u.r));
  auto routed = [&](A16Args a) {
    a.ids = c.ids, a.weights = c.weights, a.b = c.b, a.k = c.k, a.count = static_cast<int>(c.e->count);
    return a;
  };
  cudaError_t e = cudaSuccess;
  if (u.r > 0) {
    A16Args a = routed(product(u.l1q, u.sl1, nullptr, u.m, u.r, 0));
    a.x = c.x, a.ldx = c.ldx, a.out = h1;
    e = launch_rows<kModeH, 1, true>(a, c.b, pairs, st);
    if (e != cudaSuccess) return e;
  }
  {
    A16Args a = routed(product(u.rq, u.sr, u.l2t, u.m, u.n, u.r));
    a.x = c.x, a.ldx = c.ldx, a.h = h1, a.f = static_cast<int>(f), a.out = act, a.out_lo = act_lo;
    a.tiles = static_cast<int>(f / 16);
    a.ids_ready = a.x_ready = u.r > 0;
    e = launch_rows<kModeAct, 1, true>(a, c.b, pairs, st);
    if (e != cudaSuccess) return e;
  }
  if (d.r > 0) {
    A16Args a = routed(product(d.l1q, d.sl1, nullptr, d.m, d.r, 0));
    a.x = act, a.x_lo = act_lo, a.ldx = f, a.out = h2;
    a.ids_ready = true;
    e = launch_rows<kModeH, 2, true>(a, c.b, pairs, st);
    if (e != cudaSuccess) return e;
  }
  A16Args a = routed(product(d.rq, d.sr, d.l2t, d.m, d.n, d.r));
  a.x = act, a.x_lo = act_lo, a.ldx = f, a.h = h2, a.base = c.base, a.out = c.y;
  a.ids_ready = true, a.x_ready = d.r > 0;
  return launch_rows<kModeY, 2, true>(a, c.b, pairs, st);
}

}  // namespace twq
