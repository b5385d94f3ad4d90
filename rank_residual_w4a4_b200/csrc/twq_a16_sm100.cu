// Products of few rows of BF16 activations with packed 4-bit weights: the layer itself for up to
// 64 tokens, and the gated products of the experts that a router chose.
//
// A group's sum over its 128 codes is taken exactly as in the quantized layer, only that the other
// operand is BF16: codes are small integers, which BF16 holds, so mma.sync m16n8k16 multiplies them
// exactly and sums in fp32, and the group's fp32 scale multiplies that sum once.
//
// A block takes 256 or 128 weight columns (the M side of the products; rows of activations are the N
// side, 8 to a tile) and walks the reduction in steps of two groups through a ring in shared memory:
//   TMA warp   the step's codes, 128 bytes of each column in the 128-byte swizzle, and scales
//   X warps    the step's activations, gathered, in the order in which the products take them
//   8, 4 warps products, 32 columns each
// A cluster of blocks splits the reduction where there are few columns, and adds up over distributed
// shared memory in a fixed order.
//
// 16 bytes (32 codes) of a column go to one lane. The order in which a lane's codes go through the
// products is free as long as the activations follow it: codes i and i + 4 of a word become one BF16
// pair by one logic operation (0x4300 | (code ^ 8) is 136 + code) and one exact subtraction. That
// conversion, 11 instructions for 8 codes, is most of a warp's some 240 instructions for 32 columns
// x one group; at the measured copy rate (6.55 TB/s) a quarter of an SM has 386 cycles for them. The
// low-rank factor L2 comes last, in steps of 64 ranks.
//
// What bounds it, in cycles (1965 MHz) that a quarter of an SM takes for 32 columns x one group, from the
// difference of 4096 x 151552 and 4096 x 75776, so without start and end:
//     rows                                                    8     16     32
//     as it runs, blocks and warps as planned               472    620   1108   (64: twice 32)
//     the same with nothing multiplied                      435    407    599
//     products alone, 4 | 2 | 1 warps, operands there   323 | 355 | 412
// Up to 8 rows it is the copies as they are made (5.8 TB/s with nothing multiplied; two slots in the ring,
// since two blocks and their parts share an SM), and the products add 8% to them: 5.4 TB/s. Start, first
// copies, joining and end are 3.7 us more: 18.5 us for 4096 x 37888 (82 MB), 10.1 for 4096 x 14336 with 4 rows.
// From 9 rows on it is the products: two tiles of 8 rows, and with 32 rows 64 mma.sync of 8 cycles each, while
// the sums of so many rows leave 2 warps a quarter, and X is staged by every block (599 above): 28.9 us for 32
// rows of 5120 x 18944. Small layers are bound by two launches, first copies and joining: 7.4 us for one row
// of 4096 x 4096 with rank 128.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "sm100_ptx.cuh"
#include "twq_a16.h"
#include "twq_adapter.h"
#include "twq_internal.h"

namespace twq {

__device__ int g_a16_status;

namespace {

constexpr int kBox = 128;                 // weight columns of a copy, at most
constexpr int kYStride = 36;              // floats between the rows of a warp's sums
constexpr int kSms = 148;
constexpr int kMaxSlots = 4;
constexpr int kMaxSmem = 226 * 1024;      // dynamic

enum Mode : int {
  kModeH = 0,    // h = bf16(x D(L1))
  kModeAct = 1,  // a = silu(g) u, in two BF16 terms
  kModeY = 2,    // y = x D(R) + h L2
  kModePart = 3, // the same in fp32, not rounded
};

// Site codes of the bounded waits.
enum : int { kSiteEmpty = 71, kSiteXEmpty, kSiteWFull, kSiteXFull, kSiteSums, kSiteLand };

struct A16Args {
  CUtensorMap wq, ws, wl;  // codes, scales, L2: the experts' rows one after another
  const uint8_t* q;        // what the maps are of (host)
  const float* s;
  const uint16_t* l2t;
  int K, n, r;             // r: ranks of L2 read here
  int f;                   // kModeAct: gate columns (n = 2 f)
  int width;               // columns of a box (kModeAct: gates in one, what they multiply in the other)
  const uint16_t* x;       // token rows (row stride ldx), or the pairs' activations
  const uint16_t* x_lo;    // kParts == 2: the activations' second terms
  int64_t ldx;
  const uint16_t* h;       // low-rank input, tokens or pairs x r
  const int32_t* ids;      // b x k
  int b, k, count;
  uint16_t* out;           // kModePart: fp32
  uint16_t* out_lo;        // kModeAct
  int blocks;              // blocks of columns
  int split_log;           // log2 of the blocks of a cluster
  int slots;               // of the ring
  int parts;               // room for other blocks' parts of a job
  bool ids_ready, x_ready; // complete before this kernel starts, whatever it waits for
  uint64_t wait_ns;
  int stall;               // self-test: a block's last step gets no activations
};

struct WaitState {  // a block's, in shared memory
  int gave_up;
  uint64_t ns;  // limit of a wait
};
// That limit, for block `rank` of a cluster. In the self-test each outlasts those in front of it.
__host__ __device__ inline uint64_t wait_limit(uint64_t ns, bool stall, int rank) { return stall ? ns * (rank + 1) : ns; }
// The limit for peers' parts, of a block with `steps` steps. A peer may store into a block only while that is
// there, so it is longer than any peer takes to send: one has a step more at most, and in each waits at most
// twice, for weights and for activations, up to its own limit, at most the last block's. (Once a wait has run out it
// waits no more, but walks on and sends.) The rest of a step, under 1 us, is counted at 0.1 ms, and 2 s are added.
__host__ __device__ inline uint64_t parts_limit(uint64_t ns, bool stall, int split, int steps) {
  return (2 * wait_limit(ns, stall, split - 1) + 100000) * (steps + 1) + 2000000000ull;
}
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile WaitState* w, int site) {
  const uint64_t t0 = global_timer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (w->gave_up) return false;
    if (global_timer_ns() - t0 > w->ns) {
      atomicCAS(&g_a16_status, 0, site);
      w->gave_up = 1;
      return false;
    }
  }
}
// The same on an address.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Bounded wait of a warp: one answer for all of its lanes; false once the block is giving up.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile WaitState* w, int site) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xFFFFFFFFu, wait_slow(bar, parity, w, site));
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
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
// What may be read before this kernel's own wait: written by a kernel further in front, for whose end the one
// in front has waited before it let this one start (ids_ready, x_ready). It lies in L2 then, but nothing has
// told this SM's L1 so. Single words are read by loads that are strong at the GPU's scope, which L1 does not
// serve; rows of activations by plain ones behind an acquire at that scope, from which on L1 holds nothing from
// before. (Strong loads of rows fetch each 32-byte sector twice: 32 rows of 5120 x 18944 took 31.7 us, not 28.8.)
__device__ __forceinline__ void acquire_early(const uint16_t* p) {
  asm volatile("{\n\t.reg .b32 v;\n\tld.acquire.gpu.global.b32 v, [%0];\n\t}" ::"l"(p) : "memory");
}
__device__ __forceinline__ uint32_t ld4_early(const void* p) {
  uint32_t v;
  asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld8(const void* p) {
  uint2 v;
  asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
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

// The jobs [job0, job1) of a cluster, `per` steps each, and its blocks' shares of their steps, counted from job0's
// first.
struct Shares {
  int job0, job1, total;
  const int& split_log;
  __host__ __device__ Shares(int jobs, int clusters, int cluster, int per, const int& log) : split_log(log) {
    const int each = jobs / clusters, more = jobs - each * clusters;  // `more` clusters have one more
    job0 = each * cluster + (cluster < more ? cluster : more), job1 = job0 + each + (cluster < more);
    total = (job1 - job0) * per;
  }
  __host__ __device__ int begin(int rank) const { return total * rank >> split_log; }
  __host__ __device__ bool any(int rank) const { return begin(rank) < begin(rank + 1); }
  // The block that began the job whose first step is `first`, of which `rank` has a later one as its own first.
  __host__ __device__ int owner(int rank, int first) const {
    int o = rank - 1;
    while (begin(o) > first) --o;
    return o;
  }
  // f(whether it has steps) for each block behind `rank` up to the last that goes on with a job that ends at `end`.
  template <typename F>
  __host__ __device__ void others(int rank, int end, F f) const {
    for (int r = rank + 1; r < 1 << split_log && begin(r) < end; ++r) f(any(r));
  }
};

// What of a block's shared memory is where, in bytes from a 1024-byte boundary.
struct Layout {
  int sums, recv, chunks, order, cnt, before, total;
};

// kWarps: that multiply, 32 weight columns each. kModeH, whose columns are few: two warps have the same
// columns and one group of a step each.
template <int kWarps, int NT, int kMode, int kParts, bool kRouted>
struct Kernel {
  static constexpr int kShare = kMode == kModeH ? 2 : 1;
  static constexpr int kMulThreads = kWarps * 32, kCols = kWarps / kShare * 32;
  // Copies of a step: of 128 columns, or of the block's (kModeAct: of half, gates and what they multiply).
  static constexpr int kBoxCols = kMode == kModeAct ? kCols / 2 : kCols < kBox ? kCols : kBox;
  static constexpr int kWBytes = kCols * 128, kSBytes = kCols * 8 < 1024 ? 1024 : kCols * 8;
  static constexpr int kCap = 8 * NT / kParts;                 // rows of activations in a chunk
  static constexpr int kXWarps = NT == 1 ? 2 : 3;
  static constexpr int kThreads = kMulThreads + 32 + 32 * kXWarps;
  static constexpr int kBlocksPerSm = (kWarps == 8 ? 1 : 2) + (NT == 1);
  static constexpr int kSlot = kWBytes + kSBytes + 4096 * NT;

  static __host__ __device__ int max_chunks(int pairs, int count) {
    const int groups = pairs < count ? pairs : count;
    return groups + pairs / kCap < pairs ? groups + pairs / kCap : pairs;
  }
  // parts: other blocks' parts of a job that there is room for.
  static __host__ __device__ Layout layout(int b, int k, int count, int slots, int parts) {
    const int pairs = kRouted ? b * k : b;
    Layout l;
    l.sums = slots * kSlot;
    l.recv = l.sums + kWarps * kCap * kYStride * 4;
    l.chunks = l.recv + parts * kCap * kCols * 4;
    l.order = l.chunks + (kRouted ? max_chunks(pairs, count) * 8 : 0);
    l.cnt = l.order + (kRouted ? (pairs * 2 + 7) / 8 * 8 : 0);
    l.total = (l.cnt + (kRouted ? count * 4 : 0) + 15) / 16 * 16;
    // Of many pairs: beside the rest where it does not fit into the ring, which is used after it.
    const int ranks = kRouted && pairs > 32 ? (pairs + 31) / 32 * count * 2 : 0;
    l.before = ranks <= slots * kSlot && slots > 0 ? 0 : l.total;
    l.total += l.before ? (ranks + 15) / 16 * 16 : 0;
    return l;
  }
};

// Chunks of at most `cap` rows that share an expert, experts ascending, rows of an expert in the
// order of their pairs: {expert, first place in `order` | rows << 16}. Returns their number.
__device__ __noinline__ int make_chunks(const int32_t* ids, int pairs, int count, int cap, uint2* chunk,
                                        uint16_t* order, int* cnt, uint16_t* before, int* number) {
  if (pairs <= 32) {  // in one warp's registers
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      const unsigned lower = (1u << lane) - 1u, all = 0xFFFFFFFFu;
      int id = lane < pairs ? static_cast<int>(ld4_early(ids + lane)) : -1;
      if (id < 0 || id >= count) id = -1;
      const unsigned same = __match_any_sync(all, id);
      const bool leads = id >= 0 && !(same & lower);
      int place = 0, at = 0;  // of the leader's expert: rows and chunks of the experts before it
      for (unsigned todo = __ballot_sync(all, leads); todo; todo &= todo - 1) {
        const int l = __ffs(todo) - 1;
        const int e = __shfl_sync(all, id, l), n = __popc(__shfl_sync(all, same, l));
        if (e < id) place += n, at += (n + cap - 1) / cap;
      }
      if (leads)
        for (int i = 0, n = __popc(same); i < n; i += cap)
          chunk[at + i / cap] = make_uint2(id, (place + i) | (min(cap, n - i) << 16));
      if (id >= 0) order[place + __popc(same & lower)] = static_cast<uint16_t>(lane);
      const int chunks = __reduce_add_sync(all, leads ? (__popc(same) + cap - 1) / cap : 0);
      if (lane == 0) *number = chunks;
    }
    __syncthreads();
    return *number;
  }
  // More: each warp ranks the pairs of some segments of 32 among themselves; `before`, segments x count,
  // then has how many pairs of an expert the segments before one hold.
  constexpr int kMine = (kA16MaxRows * kMoeMaxChoices / 32 + 4) / 5;  // segments of a warp, of 5 warps or more
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int segments = (pairs + 31) >> 5;
  int id[kMine], rank[kMine];
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int at = (warp + j * warps) * 32 + lane;
    id[j] = at < pairs ? static_cast<int>(ld4_early(ids + at)) : -1;
    if (id[j] >= count) id[j] = -1;
  }
  for (int i = tid; i < segments * count; i += blockDim.x) before[i] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int at = warp + j * warps;
    if (at >= segments) break;
    const unsigned same = __match_any_sync(0xFFFFFFFFu, id[j] < 0 ? -1 : id[j]);
    rank[j] = __popc(same & ((1u << lane) - 1u));
    if (id[j] >= 0 && rank[j] == 0) before[at * count + id[j]] = static_cast<uint16_t>(__popc(same));
  }
  __syncthreads();
  for (int e = tid; e < count; e += blockDim.x) {
    int n = 0;
    for (int i = 0; i < segments; ++i) {
      const int here = before[i * count + e];
      before[i * count + e] = static_cast<uint16_t>(n);
      n += here;
    }
    cnt[e] = n;
  }
  __syncthreads();
  if (warp == 0) {
    int rows = 0, chunks = 0;
    for (int e0 = 0; e0 < count; e0 += 32) {
      const int e = e0 + lane;
      const int c = e < count ? cnt[e] : 0;
      if (!__any_sync(0xFFFFFFFFu, c)) continue;
      const int n = (c + cap - 1) / cap;
      int both = c | n << 16;  // up to 1024 of each
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, both, d);
        if (lane >= d) both += o;
      }
      const int first = rows + (both & 0xFFFF) - c, at = chunks + (both >> 16) - n;
      if (c) cnt[e] = first;
      for (int i = 0; i < n; ++i)
        chunk[at + i] = make_uint2(e, (first + i * cap) | (min(cap, c - i * cap) << 16));
      both = __shfl_sync(0xFFFFFFFFu, both, 31);
      rows += both & 0xFFFF;
      chunks += both >> 16;
    }
    if (lane == 0) *number = chunks;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int at = warp + j * warps;
    if (at < segments && id[j] >= 0)
      order[cnt[id[j]] + before[at * count + id[j]] + rank[j]] = static_cast<uint16_t>(at * 32 + lane);
  }
  fence_proxy_async_smem();  // `before` may be the ring's
  __syncthreads();
  return *number;
}

template <int kWarps, int NT, int kMode, int kParts, bool kRouted>
__global__ void __launch_bounds__(Kernel<kWarps, NT, kMode, kParts, kRouted>::kThreads,
                                  Kernel<kWarps, NT, kMode, kParts, kRouted>::kBlocksPerSm)
    a16_kernel(const __grid_constant__ A16Args a) {
  using K = Kernel<kWarps, NT, kMode, kParts, kRouted>;
  constexpr int kCap = K::kCap, kSlot = K::kSlot, kCols = K::kCols, kMulThreads = K::kMulThreads;
  constexpr int kWBytes = K::kWBytes, kSBytes = K::kSBytes, kBoxCols = K::kBoxCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
  __shared__ uint64_t s_wfull[kMaxSlots], s_xfull[kMaxSlots], s_empty[kMaxSlots];
  __shared__ uint64_t s_recv;
  __shared__ WaitState s_wait;
  __shared__ int s_chunks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int split = 1 << a.split_log;
  const int rank = blockIdx.x & (split - 1), cluster = blockIdx.x >> a.split_log;
  const Layout lay = K::layout(a.b, a.k, a.count, a.slots, a.parts);
  uint2* const s_chunk = reinterpret_cast<uint2*>(smem + lay.chunks);
  uint16_t* const s_order = reinterpret_cast<uint16_t*>(smem + lay.order);

  if (tid == 0) {
    for (int i = 0; i < a.slots; ++i) {
      mbar_init(&s_wfull[i], 1);
      mbar_init(&s_xfull[i], 1);
      mbar_init(&s_empty[i], kWarps);
    }
    mbar_init(&s_recv, 1);
    fence_barrier_init();
    s_wait.gave_up = 0;
    s_wait.ns = wait_limit(a.wait_ns, a.stall, rank);
  }
  if (!a.ids_ready) {
    pdl_wait();
    pdl_launch_dependents();
  }
  int chunks = 1;
  if constexpr (kRouted) {
    chunks = make_chunks(a.ids, a.b * a.k, a.count, kCap, s_chunk, s_order, reinterpret_cast<int*>(smem + lay.cnt),
                         reinterpret_cast<uint16_t*>(smem + lay.before), &s_chunks);
  } else {
    chunks = (a.b + kCap - 1) / kCap;
    __syncthreads();
  }
  if (split > 1) cluster_arrive_relaxed();  // this block's barriers exist
  auto chunk_expert = [&](int c) { return kRouted ? static_cast<int>(s_chunk[c].x) : 0; };
  auto chunk_first = [&](int c) { return kRouted ? static_cast<int>(s_chunk[c].y & 0xFFFFu) : c * kCap; };
  auto chunk_rows = [&](int c) {
    return kRouted ? static_cast<int>(s_chunk[c].y >> 16) : min(kCap, a.b - c * kCap);
  };
  auto pair_of = [&](int first, int i) { return kRouted ? static_cast<int>(s_order[first + i]) : first + i; };

  // The work. A job is a chunk and a block of columns (chunks of one block next to one another where
  // they share the weights). A cluster has the jobs [job0, job1), and each of its blocks an equal share
  // [lo, hi) of their steps, one job after the other: so a block may end a job that the one before it
  // began. All roles walk the same steps.
  const int groups = a.K >> 7, code_steps = (groups + 1) / 2, per = code_steps + (a.r + 63) / 64;
  const int jobs = chunks * a.blocks, clusters = gridDim.x >> a.split_log;
  const Shares shares(jobs, clusters, cluster, per, a.split_log);
  const int job1 = shares.job1, lo = shares.begin(rank), hi = shares.begin(rank + 1);
  struct Walk {
    int job, block, chunk, u;  // step u of the job
  };
  auto enter_job = [&](Walk& k) {
    if constexpr (kRouted)
      k.chunk = k.job / a.blocks, k.block = k.job - k.chunk * a.blocks;
    else
      k.block = k.job / chunks, k.chunk = k.job - k.block * chunks;
  };
  Walk at0 = {shares.job0, 0, 0, 0};
  if (lo < hi) {
    const int skip = lo / per;
    at0.job += skip, at0.u = lo - skip * per;
    enter_job(at0);
  }
  // The next step; true where it is of another job.
  auto advance = [&](Walk& k) {
    if (++k.u < per) return false;
    ++k.job, k.u = 0;
    if (k.job < job1) enter_job(k);
    return true;
  };
  struct Turn {
    int slot = 0;
    uint32_t phase = 0;
  };
  auto next_slot = [&](Turn& s) {
    if (++s.slot == a.slots) s.slot = 0, s.phase ^= 1;
  };

  if (warp == kWarps) {  // TMA
    Turn s;
    Walk k = at0;
    int issued = 0;
    for (int v = lo; v < hi; ++v) {
      // The slot is free, and what was loaded into it is there (products that gave up do not wait for that).
      if (issued >= a.slots && !(wait(&s_empty[s.slot], s.phase ^ 1, &s_wait, kSiteEmpty) &&
                                 wait(&s_wfull[s.slot], s.phase ^ 1, &s_wait, kSiteWFull)))
        break;
      if (lane == 0) {
        const int col = k.block * (kMode == kModeAct ? kCols / 2 : kCols);
        const int boxes = kMode == kModeAct ? 2 : min(kCols / kBoxCols, (a.n - col + kBoxCols - 1) / kBoxCols);
        const int next = kMode == kModeAct ? a.f : kBoxCols;  // from one box to the other
        uint8_t* const dst = smem + s.slot * kSlot;
        const int e = chunk_expert(k.chunk), row = e * a.n + col;
        if (k.u < code_steps) {
          mbar_arrive_expect_tx(&s_wfull[s.slot], boxes * a.width * (128 + 8));
#pragma unroll 1
          for (int i = 0; i < boxes; ++i) {
            tma_load_2d(dst + i * kBoxCols * 128, &a.wq, &s_wfull[s.slot], k.u * 128, row + i * next);
            tma_load_2d(dst + kWBytes + i * kBoxCols * 8, &a.ws, &s_wfull[s.slot], col + i * next,
                        e * groups + 2 * k.u);
          }
        } else {
          mbar_arrive_expect_tx(&s_wfull[s.slot], boxes * a.width * 128);
#pragma unroll 1
          for (int i = 0; i < boxes; ++i)
            tma_load_2d(dst + i * kBoxCols * 128, &a.wl, &s_wfull[s.slot], (k.u - code_steps) * 64, row + i * next);
        }
      }
      __syncwarp();
      ++issued;
      next_slot(s);
      advance(k);
    }
    // No copy is in flight when the block leaves, whether it was used or the block gave up.
    if (lane == 0) {
      for (int i = max(0, issued - a.slots); i < issued; ++i) {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(&s_wfull[i % a.slots], (i / a.slots) & 1)) {
          if (global_timer_ns() - t0 > 2000000000ull) {
            atomicExch(&g_a16_status, kSiteLand);
            break;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp > kWarps) {
    // Activations, each warp a step in turn, its next one's on their way meanwhile. No more warps than
    // slots: one that does not wait at the steps of the others must not get two turns of the ring ahead.
    const int turns = min(K::kXWarps, a.slots), turn = warp - kWarps - 1;
    if (a.x_ready)
      acquire_early(a.x);
    else
      pdl_wait();
    if (a.ids_ready) pdl_launch_dependents();
    constexpr int kN = NT < 2 ? 1 : 2;  // tiles whose loads are in flight together
    bool waited = !a.x_ready;
    Turn s;
    Walk k = at0;
    int v = lo, rows = 0, first = 0, known = -1;
    const uint16_t* row[NT];  // of the lane's column of each tile
    uint4 x[kN][2][4];
    // Loads of tiles n0 and, if there is one, n0 + 1 of the step.
    auto load = [&](int n0) {
#pragma unroll
      for (int nt = 0; nt < kN; ++nt) {
        if (nt > 0 && (n0 + nt) * 8 >= rows * kParts) break;
        const uint16_t* const from = row[NT <= 2 ? nt : n0 + nt] + k.u * 256;
#pragma unroll
        for (int w = 0; w < 2; ++w)
          if (w == 0 || 2 * k.u + 1 < groups) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[nt][w][j] = ld16(from + w * 128 + j * 8);
          }
      }
    };
    auto begin = [&] {  // the step's chunk, and its first loads
      if (v >= hi) return;
      if (known != k.chunk) {
        known = k.chunk;
        first = chunk_first(k.chunk), rows = chunk_rows(k.chunk);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int c = nt * 8 + g, i = kParts == 2 ? c >> 1 : c;
          // columns beyond the rows: the first row's, into sums that no one reads
          const int pr = pair_of(first, i < rows ? i : 0);
          const int64_t at = kRouted && kParts == 1 ? pr / a.k : pr;
          row[nt] = (kParts == 2 && (c & 1) ? a.x_lo : a.x) + at * a.ldx + t * 32;
        }
      }
      if (k.u < code_steps) load(0);
    };
    auto skip = [&](int by) {
#pragma unroll 1
      for (int i = 0; i < by && v < hi; ++i) {
        ++v;
        next_slot(s);
        advance(k);
      }
    };
    if (turn >= turns) v = hi;
    skip(turn);
    begin();
    while (v < hi) {
      if (a.stall && v + 1 == hi) break;
      uint8_t* const dst = smem + s.slot * kSlot + kWBytes + kSBytes + lane * 16;
      if (k.u >= code_steps) {
        if (!waited) pdl_wait();
        waited = true;
      }
      if (v - lo >= a.slots && !wait(&s_empty[s.slot], s.phase ^ 1, &s_wait, kSiteXEmpty)) break;
      if (k.u < code_steps) {
#pragma unroll
        for (int n0 = 0; n0 < NT; n0 += kN) {
          if (n0 > 0) {
            if (n0 * 8 >= rows * kParts) break;
            load(n0);
          }
#pragma unroll
          for (int nt = 0; nt < kN; ++nt) {
            if (nt > 0 && (n0 + nt) * 8 >= rows * kParts) break;
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint4 v4 = x[nt][w][j];
                *reinterpret_cast<uint4*>(dst + (w * NT + n0 + nt) * 2048 + j * 512) =
                    make_uint4(__byte_perm(v4.x, v4.z, 0x5410), __byte_perm(v4.x, v4.z, 0x7632),
                               __byte_perm(v4.y, v4.w, 0x5410), __byte_perm(v4.y, v4.w, 0x7632));
              }
          }
        }
      } else {  // h: ranks as they lie, zeros beyond them
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int c = nt * 8 + g, i = kParts == 2 ? c >> 1 : c;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int at = (k.u - code_steps) * 64 + w * 32 + t * 8;
            uint4 v4 = make_uint4(0, 0, 0, 0);
            if (i < rows && !(kParts == 2 && (c & 1)) && at < a.r)
              v4 = ld16(a.h + static_cast<int64_t>(pair_of(first, i)) * a.r + at);
            *reinterpret_cast<uint4*>(dst + (w * NT + nt) * 512) = v4;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_xfull[s.slot]);
      skip(turns);
      begin();
    }
  } else {  // products
    float* const sums = reinterpret_cast<float*>(smem + lay.sums);
    float* const mine = sums + warp * kCap * kYStride;
    // The lane's columns: sigma + 8 i of its warp's 32, i < 4 (kModeAct: of its 16 gates for i < 2, else
    // of what they multiply). sigma orders them so that 8 lanes read 128 bytes without conflict.
    const int sigma = (g & 1) * 4 + (g >> 1);
    const int wr = warp % (kWarps / K::kShare), wk0 = warp / (kWarps / K::kShare);  // columns, group of a step
    const int line = kMode == kModeAct ? wr * 16 + sigma : wr * 32 + sigma;
    auto line_of = [&](int i) { return kMode == kModeAct ? (i & 1) * 8 + (i >> 1) * kBoxCols : i * 8; };
    // Offsets into a slot, of 32 bits.
    const uint32_t base = static_cast<uint32_t>(smem - smem_raw);
    const uint32_t w_at[2] = {line * 128u + ((t ^ sigma) << 4), line * 128u + (((4 + t) ^ sigma) << 4)};
    const uint32_t s_at = kWBytes + line / kBoxCols * kBoxCols * 8 + line % kBoxCols * 4, s_next = a.width * 4;
    const uint32_t x_at = kWBytes + kSBytes + lane * 16;
    auto lds16 = [&](uint32_t at) { return *reinterpret_cast<const uint4*>(smem_raw + at); };
    auto barrier = [&] { asm volatile("bar.sync 1, %0;" ::"n"(kMulThreads) : "memory"); };

    auto add4 = [](float4& o, const float4& p) { o.x += p.x, o.y += p.y, o.z += p.z, o.w += p.w; };

    // Outputs are made in items of four neighbours (kModeAct: of four gates and what they multiply,
    // 16 columns on) of one row.
    constexpr int kItems = kMode == kModeAct ? kCols / 8 : kCols / 4, kQuads = kMode == kModeAct ? 2 : 1;
    auto sum_of = [&](int item, int q) {  // this block's
      const int c = item % kItems, col = kMode == kModeAct ? (c >> 2) * 32 + (c & 3) * 4 + 16 * q : c * 4;
      const float* const at = sums + ((col >> 5) * kCap + item / kItems) * kYStride + (col & 31);
      float4 o = *reinterpret_cast<const float4*>(at);
      if constexpr (K::kShare == 2) add4(o, *reinterpret_cast<const float4*>(at + kWarps / 2 * kCap * kYStride));
      return o;
    };
    auto put_item = [&](int block, int first, int item, const float4 (&v)[kQuads]) {
      const int row = item / kItems, c = item % kItems;
      const int64_t line = pair_of(first, row);
      if constexpr (kMode == kModeAct) {
        if (block * (kCols / 2) + c * 4 >= a.f) return;
        const float4 gate = v[0], up = v[1];
        const float act[4] = {gate.x / (1.0f + expf(-gate.x)) * up.x, gate.y / (1.0f + expf(-gate.y)) * up.y,
                              gate.z / (1.0f + expf(-gate.z)) * up.z, gate.w / (1.0f + expf(-gate.w)) * up.w};
        // a in two BF16 terms, 2^-17 of a off at most, since mma.sync takes BF16 beside the codes: each is a column
        // of the down product, 4 rows to a tile. A third term would leave 2 rows to a tile, for an error that y's
        // own rounding (2^-8) hides as it is: against 64 bits y's error is that of the exact y, rounded (0.0016 to
        // 0.0017), and 1 to 4 of a thousand elements of y are the neighbour of that.
        float left[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float o = __bfloat162float(__float2bfloat16_rn(act[e]));
          left[e] = isfinite(o) ? act[e] - o : 0.0f;
        }
        const int64_t at = line * a.f + block * (kCols / 2) + c * 4;
        *reinterpret_cast<uint2*>(a.out + at) = make_uint2(pack2(act[0], act[1]), pack2(act[2], act[3]));
        *reinterpret_cast<uint2*>(a.out_lo + at) = make_uint2(pack2(left[0], left[1]), pack2(left[2], left[3]));
      } else {
        const int col = block * kCols + c * 4;
        if (col >= a.n) return;
        const float4 o = v[0];
        const int64_t at = line * a.n + col;
        if constexpr (kMode == kModePart)
          *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = o;
        else
          *reinterpret_cast<uint2*>(a.out + at) = make_uint2(pack2(o.x, o.y), pack2(o.z, o.w));
      }
    };
    float acc[2][NT][4];
    auto clear = [&] {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][nt][j] = 0.0f;
    };
    // Stores the sums to the warp's own rows.
    auto leave = [&](int rows) {
      auto put = [&](int i, float v0, float v1, float v2, float v3) {
        if (i >= rows) return;
        float* const y = mine + i * kYStride + sigma;
        y[0] = v0, y[8] = v1, y[16] = v2, y[24] = v3;
      };
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
      clear();
    };

    // A block's part of a job that another one began goes to that one, as its (rank - owner - 1)-th part.
    const int rest = lo < hi ? hi % per : 0;  // steps of the last job, if it goes on
    float4* const recv = reinterpret_cast<float4*>(smem + lay.recv);
    constexpr int kPart = kCap * kItems * kQuads;  // of one block, in quads
    auto send_part = [&](int rows) {
      const int owner = shares.owner(rank, lo - at0.u);
      cluster_wait_acquire();  // the owner's barrier exists
      const uint32_t to = map_peer(smem_u32(recv + (rank - owner - 1) * kPart), owner);
      const uint32_t bar = map_peer(smem_u32(&s_recv), owner);
#pragma unroll 1
      for (int i = tid; i < rows * kItems; i += kMulThreads)
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
          const float4 o = sum_of(i, q);
          st_async_peer_v4(to + (i * kQuads + q) * 16, o.x, o.y, o.z, o.w, bar);
        }
    };
    // What peers store into this block lands before it leaves, whether it or they gave up: the limit is longer
    // than a peer takes to send. The stores are other blocks': an acquire at the cluster's scope orders them.
    auto wait_parts = [&] {
      const uint64_t t0 = global_timer_ns(), ns = parts_limit(a.wait_ns, a.stall, split, hi - lo);
      while (!mbar_try_wait_cluster(&s_recv, 0)) {
        if (global_timer_ns() - t0 > ns) {
          atomicCAS(&g_a16_status, 0, kSiteSums);
          break;
        }
      }
      __syncwarp();
    };

    // One group of 32 columns; one 32 ranks of their low-rank factors.
    int tiles = 1;  // of rows in use
    auto code_unit = [&](uint32_t at, int wk) {
      uint4 w[4];
      float sc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = lds16(at + (wk ? w_at[1] : w_at[0]) + line_of(i) * 128);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sc[i] = *reinterpret_cast<const float*>(
            smem_raw + (at + s_at + wk * s_next + (kMode == kModeAct ? (i & 1) * 32 + (i >> 1) * kBoxCols * 8 : i * 32)));
      float d[2][NT][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t c[2][2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 w0 = w[2 * i], w1 = w[2 * i + 1];
          const uint32_t a0 = j == 0 ? w0.x : j == 1 ? w0.y : j == 2 ? w0.z : w0.w;
          const uint32_t a1 = j == 0 ? w1.x : j == 1 ? w1.y : j == 2 ? w1.z : w1.w;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            c[i][h][0] = codes2(a0 >> (8 * h)), c[i][h][1] = codes2(a1 >> (8 * h));
            c[i][h][2] = codes2(a0 >> (8 * h + 4)), c[i][h][3] = codes2(a1 >> (8 * h + 4));
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (nt > 0 && nt >= tiles) break;
          const uint4 x = lds16(at + x_at + (wk * NT + nt) * 2048 + j * 512);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (j == 0)
              mma16816_first(d[i][nt], c[i][0][0], c[i][0][1], c[i][0][2], c[i][0][3], x.x, x.y);
            else
              mma16816(d[i][nt], c[i][0][0], c[i][0][1], c[i][0][2], c[i][0][3], x.x, x.y);
            mma16816(d[i][nt], c[i][1][0], c[i][1][1], c[i][1][2], c[i][1][3], x.z, x.w);
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt > 0 && nt >= tiles) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          acc[i][nt][0] = fmaf(sc[2 * i], d[i][nt][0], acc[i][nt][0]);
          acc[i][nt][1] = fmaf(sc[2 * i], d[i][nt][1], acc[i][nt][1]);
          acc[i][nt][2] = fmaf(sc[2 * i + 1], d[i][nt][2], acc[i][nt][2]);
          acc[i][nt][3] = fmaf(sc[2 * i + 1], d[i][nt][3], acc[i][nt][3]);
        }
      }
    };
    auto rank_unit = [&](uint32_t at, int wk) {
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = lds16(at + (wk ? w_at[1] : w_at[0]) + line_of(i) * 128);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 x = lds16(at + x_at + (wk * NT + nt) * 512);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mma16816(acc[i][nt], w[2 * i].x, w[2 * i + 1].x, w[2 * i].y, w[2 * i + 1].y, x.x, x.y);
          mma16816(acc[i][nt], w[2 * i].z, w[2 * i + 1].z, w[2 * i].w, w[2 * i + 1].w, x.z, x.w);
        }
      }
    };
    const uint32_t empty0 = smem_u32(s_empty), wfull0 = smem_u32(s_wfull), xfull0 = smem_u32(s_xfull);
    uint32_t slot = 0, phase = 0;
    bool ok = true;
    // A block that gives up walks on, so that all its warps meet at the barriers below.
    auto step_begin = [&] {
      if (!__all_sync(0xFFFFFFFFu, try_wait(wfull0 + slot * 8, phase) && try_wait(xfull0 + slot * 8, phase)))
        ok = ok && wait(&s_wfull[slot], phase, &s_wait, kSiteWFull) &&
             wait(&s_xfull[slot], phase, &s_wait, kSiteXFull);
      return base + slot * kSlot;
    };
    auto step_end = [&] {
      __syncwarp();
      if (lane == 0) arrive(empty0 + slot * 8);
      if (++slot == a.slots) slot = 0, phase ^= 1;
    };

    Walk k = at0;
    int from = at0.u;  // of the job's steps, the first of this block's
    clear();
    for (int v = lo; v < hi;) {
      const int chunk = k.chunk, block = k.block, to = min(per, from + hi - v);
      const int first = chunk_first(chunk), rows = chunk_rows(chunk);
      tiles = (rows * kParts + 7) >> 3;
      // columns that are not there: nothing to do
      const bool any = kMode == kModeAct ? block * (kCols / 2) + wr * 16 < a.f : block * kCols + wr * 32 < a.n;
      int u = from;
#pragma unroll 1
      for (; u < min(to, code_steps); ++u) {
        const uint32_t at = step_begin();
        if (ok && any) {
          if constexpr (K::kShare == 2) {
            if (2 * u + wk0 < groups) code_unit(at, wk0);
          } else if constexpr (NT <= 2) {
            code_unit(at, 0);
            if (2 * u + 1 < groups) code_unit(at, 1);
          } else {  // twice the registers: not both at once
#pragma unroll 1
            for (int wk = 0; wk < min(2, groups - 2 * u); ++wk) code_unit(at, wk);
          }
        }
        step_end();
      }
#pragma unroll 1
      for (; u < to; ++u) {
        const uint32_t at = step_begin();
#pragma unroll 1
        for (int wk = 0; wk < 2; ++wk)
          if (ok && any && (u - code_steps) * 64 + wk * 32 < a.r) rank_unit(at, wk);
        step_end();
      }
      v += to - from;
      const bool over = to == per;
      if (over) {
        ++k.job;
        if (k.job < job1) enter_job(k);
      }
      leave(rows);
      barrier();
      if (from > 0) {
        send_part(rows);
      } else {
        pdl_wait();
        int parts = 0;  // of other blocks
        if (!over) {    // this block began the job, others end it
          uint32_t bytes = 0;
          shares.others(rank, hi - rest + per, [&](bool any) {
            ++parts;
            if (any) bytes += rows * kItems * kQuads * 16;
          });
          if (tid == 0) mbar_arrive_expect_tx(&s_recv, bytes);
          __syncwarp();
          wait_parts();
        }
#pragma unroll 1
        for (int i = tid; i < rows * kItems; i += kMulThreads) {
          float4 o[kQuads];
#pragma unroll
          for (int q = 0; q < kQuads; ++q) o[q] = sum_of(i, q);
#pragma unroll 1
          for (int r = 0; r < parts; ++r)
            if (shares.any(rank + 1 + r)) {
#pragma unroll
              for (int q = 0; q < kQuads; ++q) add4(o[q], recv[r * kPart + i * kQuads + q]);
            }
          put_item(block, first, i, o);
        }
      }
      from = 0;
      if (v < hi) barrier();  // the sums are read
    }
  }
  pdl_wait();  // this grid completes only after the one in front
}

// y = base + the sum of weight * part over a token's slots, in their order; four columns per thread. A kernel
// of its own, since a token's slots are different clusters' work: atomics would add in any order, and a product
// that goes token by token has too few rows a weight. Latency of one load after the other bounds it (4.6 us
// alone and cold for 4 tokens of 4096, less behind the products, whose end its start overlaps).
constexpr int kCombineThreads = 128;
__global__ void __launch_bounds__(kCombineThreads)
    combine_kernel(const float* parts, const int32_t* ids, const float* weights, int k, int count, int n,
                   const uint16_t* base, uint16_t* y) {
  const int col = (blockIdx.x * kCombineThreads + threadIdx.x) * 4;
  const int64_t token = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  if (col >= n) return;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (base) {
    const uint2 b = ld8(base + token * n + col);
    o = make_float4(lo_f(b.x), hi_f(b.x), lo_f(b.y), hi_f(b.y));
  }
  constexpr int kAhead = 4;  // slots whose loads are in flight together
  for (int s0 = 0; s0 < k; s0 += kAhead) {
    float4 p[kAhead];
    float f[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t pair = token * k + s0 + i;
      const int id = s0 + i < k ? static_cast<int>(ld4(ids + pair)) : -1;
      f[i] = 0.0f;
      p[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (id >= 0 && id < count) {
        f[i] = __uint_as_float(ld4(weights + pair));
        const uint4 v = ld16(reinterpret_cast<const uint16_t*>(parts + pair * n + col));
        p[i] = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      o.x = fmaf(f[i], p[i].x, o.x), o.y = fmaf(f[i], p[i].y, o.y), o.z = fmaf(f[i], p[i].z, o.z),
      o.w = fmaf(f[i], p[i].w, o.w);
  }
  *reinterpret_cast<uint2*>(y + token * n + col) = make_uint2(pack2(o.x, o.y), pack2(o.z, o.w));
}

// How a launch divides its jobs (about `jobs`, of `steps` each): clusters, log2 of their blocks, and
// how many blocks' parts of a job a block may get.
struct Plan {
  int64_t clusters, cost, mine;  // mine: steps of a block, at most
  int split_log, parts;
};
// The split that the busiest SM is done with first, of at most 2^most blocks; room: clusters of 1, 2, 4 and
// 8 blocks that run at once. An SM's time for a group of 32 columns goes with the warps that multiply there: the
// constants, fitted to 8 rows of 4096 x 37888, start and end included, say 410 cycles with 16 warps and 555 with 8.
// They stand for all numbers of rows, whose own curves differ (without start and end 472 and 517 for 8 rows). What
// they choose at 4096 x 37888, and one block on an SM instead: 8 rows 18.5 us, 20.4; 32 rows 40.5, 42.5; 64 rows 77.0
// either way; 16 rows 25.2, 24.3: there they choose the worse by 4%.
// Among equal splits of a long run of choices' jobs the finer one: how many jobs there are, the GPU alone
// knows, and a cluster with one job more than another costs less (24 tokens, a quarter of 8 choices each among
// 32 local experts of 4096 x 1024: 73 us instead of 77). For a short run joining the parts costs more (one
// token, 8 of 128 experts of 2048 x 768: 18.6 us, 22.0 with the finer split).
constexpr int kShortRun = 8, kLongRun = 16;
Plan plan(int64_t jobs, int64_t steps, const int* room, int per_sm, int warps, bool all_there, int most) {
  Plan best = {0, 0, 0, 0, 0};
  for (int s = 0; s <= most; ++s) {
    if (s > 0 && steps * jobs < 2 << s) break;
    const int64_t clusters = std::min<int64_t>(jobs, room[s]);
    const int64_t mine = ((jobs + clusters - 1) / clusters * steps + (1 << s) - 1) >> s;
    const int64_t at_once = std::min<int64_t>(((clusters << s) + kSms - 1) / kSms, per_sm) * warps;
    const int64_t cost = mine * at_once * (265 + 2320 / at_once);
    if (best.clusters && cost >= best.cost + (!all_there && mine >= kLongRun)) continue;
    // Blocks that a job may reach over: all where they may have no step each (which jobs there are may be
    // known on the GPU alone).
    const int64_t least = all_there ? (jobs / clusters * steps) >> s : 0;
    const int64_t others = least ? std::min<int64_t>((1 << s) - 1, (steps + least - 2) / least) : (1 << s) - 1;
    best = {clusters, cost, mine, s, static_cast<int>(others)};
  }
  return best;
}

// How many clusters of 1, 2, 4 and 8 blocks run at once, with per_sm blocks' shared memory on an SM (a cluster
// keeps within a GPC, and GPCs differ). Asked once for each kernel, device and per_sm; only answers are kept, the
// four in one word (0: not asked yet), so that calls from several threads at once need no lock. On devices beyond
// kDevices it is asked at every launch.
constexpr int kDevices = 64, kMostPerSm = 3;
using Rooms = std::atomic<uint64_t>[kDevices][kMostPerSm];
cudaError_t clusters_at_once(const void* kernel, int threads, int per_sm, Rooms& rooms, int (&room)[4]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<uint64_t>* const known = dev < kDevices ? &rooms[dev][per_sm - 1] : nullptr;
  uint64_t all = known ? known->load(std::memory_order_relaxed) : 0;
  if (!all) {
    e = allow_smem(kernel, kMaxSmem);
    if (e != cudaSuccess) return e;
    for (int s = 0; s < 4; ++s) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((8 * kSms) << s);
      cfg.blockDim = dim3(threads);
      cfg.dynamicSmemBytes = std::min(kMaxSmem, 227 * 1024 / per_sm - 1536);
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = 1 << s;
      at[0].val.clusterDim.y = 1;
      at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
      if (e != cudaSuccess) {
        cudaGetLastError();  // returned here; not a later launch's error
        return e;
      }
      all |= static_cast<uint64_t>(std::min(std::max(n, 1), 0xFFFF)) << (16 * s);
    }
    if (known) known->store(all, std::memory_order_relaxed);
  }
  for (int s = 0; s < 4; ++s) room[s] = static_cast<int>(all >> (16 * s) & 0xFFFF);
  return cudaSuccess;
}

// A launch as it fits: of the blocks on an SM and the clusters that leave a ring of two slots or more beside
// the sums and the parts, those with the least work on the busiest SM. Many experts' lists may leave a block
// of more columns no room.
constexpr int64_t kNoFit = int64_t(1) << 56;
struct Choice {
  Plan p;
  int blocks, slots;
};

template <int kWarps, int NT, int kMode, int kParts, bool kRouted>
cudaError_t choose(const A16Args& a, Choice* out) {
  using K = Kernel<kWarps, NT, kMode, kParts, kRouted>;
  static_assert(K::kBlocksPerSm <= kMostPerSm, "places of the answers");
  static Rooms rooms;
  int64_t chunks = (a.b + K::kCap - 1) / K::kCap;
  // As many different experts as so many choices among them leave on average (13 tokens, 8 each of 128 experts of
  // 2048 x 768: 68 us, 75 if planned for as many as there may be). Other numbers of them run as well.
  if (kRouted) {
    const double pairs = a.b * a.k, used = a.count * (1.0 - std::pow(1.0 - 1.0 / a.count, pairs));
    chunks = std::min<int64_t>(K::max_chunks(a.b * a.k, a.count), std::ceil(std::max(used, pairs / K::kCap)));
  }
  const int width = kMode == kModeAct ? K::kCols / 2 : K::kCols;
  const int blocks = ((kMode == kModeAct ? a.f : a.n) + width - 1) / width;
  const int64_t steps = (a.K / 128 + 1) / 2 + (a.r + 63) / 64;
  *out = {};
  out->p.cost = kNoFit;
  for (int per_sm = K::kBlocksPerSm; per_sm > 0; --per_sm) {
    int room[4];
    const cudaError_t e =
        clusters_at_once(reinterpret_cast<const void*>(a16_kernel<kWarps, NT, kMode, kParts, kRouted>), K::kThreads,
                         per_sm, rooms, room);
    if (e != cudaSuccess) return e;
    for (int most = 3; most >= 0; --most) {
      const Plan p = plan(chunks * blocks, steps, room, per_sm, kWarps, !kRouted, most);
      const int left = 227 * 1024 / per_sm - 1024 - 1536 - K::layout(a.b, a.k, a.count, 0, p.parts).total;
      if (left < 2 * K::kSlot) continue;
      if (p.cost < out->p.cost) *out = {p, blocks, std::min(kMaxSlots, left / K::kSlot)};
      break;
    }
  }
  return cudaSuccess;
}

template <int kWarps, int NT, int kMode, int kParts, bool kRouted>
cudaError_t launch_warps(A16Args a, const Choice& c, cudaStream_t st) {
  using K = Kernel<kWarps, NT, kMode, kParts, kRouted>;
  auto kernel = a16_kernel<kWarps, NT, kMode, kParts, kRouted>;
  const Plan& p = c.p;
  if (p.cost >= kNoFit) return cudaErrorInvalidValue;
  a.blocks = c.blocks, a.slots = c.slots;
  a.split_log = p.split_log, a.parts = p.parts;
  const int split = 1 << p.split_log;
  const Layout l = K::layout(a.b, a.k, a.count, a.slots, a.parts);
  a.width = std::min(K::kBoxCols, a.n);
  bool ok = encode_map_2d(&a.wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.q, a.K / 2, int64_t(a.count) * a.n, a.K / 2, 128,
                          a.width, CU_TENSOR_MAP_SWIZZLE_128B) &&
            encode_map_2d(&a.ws, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.s, a.n, int64_t(a.count) * (a.K / 128),
                          int64_t(a.n) * 4, a.width, 2, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (ok && a.r > 0)
    ok = encode_map_2d(&a.wl, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.l2t, a.r, int64_t(a.count) * a.n, a.r * 2, 64,
                       a.width, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem(kernel, kMaxSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.clusters * split));
  cfg.blockDim = dim3(K::kThreads);
  cfg.dynamicSmemBytes = l.total + 1024;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = split;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Blocks of 256 columns, or of 128 where that leaves the busiest SM less. At the same work, blocks of 128
// where a run is short: they are done sooner after their last step (one row, 4096 -> 4096 with rank 128: 7.4
// us, 8.4 with 256), and of 256 where it is longer: they stage the activations half as often (61 rows, 5120 ->
// 25600 with rank 64: 73.5 us, 82.1 with 128; 32 rows, 5120 -> 18944: 28.6, 30.6).
template <int NT, int kMode, int kParts, bool kRouted>
cudaError_t launch(const A16Args& a, cudaStream_t st) {
  Choice narrow;
  cudaError_t e = choose<4, NT, kMode, kParts, kRouted>(a, &narrow);
  if (e != cudaSuccess) return e;
  if constexpr (kMode != kModeH) {
    Choice wide;
    e = choose<8, NT, kMode, kParts, kRouted>(a, &wide);
    if (e != cudaSuccess) return e;
    if (wide.p.cost < narrow.p.cost || (wide.p.cost == narrow.p.cost && wide.p.mine >= kShortRun))
      return launch_warps<8, NT, kMode, kParts, kRouted>(a, wide, st);
  }
  return launch_warps<4, NT, kMode, kParts, kRouted>(a, narrow, st);
}

// Tiles of a chunk: for as many rows as there are, or as an expert has on average twice over (then
// most experts' weights are read once).
template <int kMode, int kParts, bool kRouted>
cudaError_t launch_rows(const A16Args& a, cudaStream_t st) {
  const int rows = kRouted ? std::min(a.b, std::max(1, 2 * a.b * a.k / a.count)) : a.b;
  if (rows * kParts <= 8) return launch<1, kMode, kParts, kRouted>(a, st);
  if (rows * kParts <= 16) return launch<2, kMode, kParts, kRouted>(a, st);
  return launch<4, kMode, kParts, kRouted>(a, st);
}

thread_local uint64_t t_stall_ns = 0;  // self-test: the calling thread's limit of the waits, or 0

// One product of `count` experts' weights.
A16Args product(const uint8_t* q, const float* s, const uint16_t* l2t, int64_t K, int64_t n, int64_t r,
                int64_t count) {
  A16Args a = {};
  a.q = q, a.s = s, a.l2t = l2t;
  a.K = static_cast<int>(K), a.n = static_cast<int>(n), a.r = static_cast<int>(r);
  a.k = 1, a.count = static_cast<int>(count);
  a.wait_ns = t_stall_ns ? t_stall_ns : 2000000000ull;
  a.stall = t_stall_ns != 0;
  return a;
}

size_t up16(size_t v) { return (v + 15) & ~size_t(15); }

}  // namespace

cudaError_t launch_a16_linear(const A16LinearCall& c, cudaStream_t st) {
  const twq_weights& w = *c.w;
  if (w.r > 0) {
    A16Args a = product(w.l1q, w.sl1, nullptr, w.m, w.r, 0, 1);
    a.x = c.x, a.ldx = c.ldx, a.b = c.b, a.out = c.h;
    a.ids_ready = true;
    const cudaError_t e = launch_rows<kModeH, 1, false>(a, st);
    if (e != cudaSuccess) return e;
  }
  A16Args a = product(w.rq, w.sr, w.l2t, w.m, w.n, w.r, 1);
  a.x = c.x, a.ldx = c.ldx, a.b = c.b, a.h = c.h, a.out = c.y;
  a.ids_ready = true, a.x_ready = w.r > 0;
  return launch_rows<kModeY, 1, false>(a, st);
}

size_t moe_workspace(int64_t pairs, const twq_experts* e) {
  return 2 * up16(2 * pairs * e->down.m) + up16(2 * pairs * e->up.r) + up16(2 * pairs * e->down.r) +
         4 * pairs * e->down.n;
}

cudaError_t launch_moe_experts(const MoeCall& c, cudaStream_t st) {
  const twq_weights &u = c.e->up, &d = c.e->down;
  const int64_t pairs = int64_t(c.b) * c.k, f = d.m;
  uint8_t* ws = static_cast<uint8_t*>(c.workspace);
  uint16_t* act = reinterpret_cast<uint16_t*>(ws);
  uint16_t* act_lo = reinterpret_cast<uint16_t*>(ws + up16(2 * pairs * f));
  uint16_t* h1 = reinterpret_cast<uint16_t*>(ws + 2 * up16(2 * pairs * f));
  uint16_t* h2 = reinterpret_cast<uint16_t*>(ws + 2 * up16(2 * pairs * f) + up16(2 * pairs * u.r));
  float* parts = reinterpret_cast<float*>(ws + 2 * up16(2 * pairs * f) + up16(2 * pairs * u.r) + up16(2 * pairs * d.r));
  // The weights `w`'s product; l1: x D(L1).
  auto routed = [&](const twq_weights& w, bool l1) {
    A16Args a = l1 ? product(w.l1q, w.sl1, nullptr, w.m, w.r, 0, c.e->count)
                   : product(w.rq, w.sr, w.l2t, w.m, w.n, w.r, c.e->count);
    a.ids = c.ids, a.b = c.b, a.k = c.k;
    return a;
  };
  cudaError_t e = cudaSuccess;
  if (u.r > 0) {
    A16Args a = routed(u, true);
    a.x = c.x, a.ldx = c.ldx, a.out = h1;
    if ((e = launch_rows<kModeH, 1, true>(a, st)) != cudaSuccess) return e;
  }
  {
    A16Args a = routed(u, false);
    a.x = c.x, a.ldx = c.ldx, a.h = h1, a.f = static_cast<int>(f), a.out = act, a.out_lo = act_lo;
    a.ids_ready = a.x_ready = u.r > 0;
    if ((e = launch_rows<kModeAct, 1, true>(a, st)) != cudaSuccess) return e;
  }
  if (d.r > 0) {
    A16Args a = routed(d, true);
    a.x = act, a.x_lo = act_lo, a.ldx = f, a.out = h2;
    a.ids_ready = true;
    if ((e = launch_rows<kModeH, 2, true>(a, st)) != cudaSuccess) return e;
  }
  {
    A16Args a = routed(d, false);
    a.x = act, a.x_lo = act_lo, a.ldx = f, a.h = h2, a.out = reinterpret_cast<uint16_t*>(parts);
    a.ids_ready = true, a.x_ready = d.r > 0;
    if ((e = launch_rows<kModePart, 2, true>(a, st)) != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((d.n / 4 + kCombineThreads - 1) / kCombineThreads), c.b);
  cfg.blockDim = dim3(kCombineThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_kernel, parts, c.ids, c.weights, c.k, static_cast<int>(c.e->count),
                            static_cast<int>(d.n), c.base, c.y);
}

void set_a16_stall(int64_t wait_limit_ns) { t_stall_ns = static_cast<uint64_t>(wait_limit_ns); }

cudaError_t read_and_clear_a16_status(int* code) {
  cudaError_t e = cudaMemcpyFromSymbol(code, g_a16_status, sizeof(int));
  if (e != cudaSuccess || *code == 0) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_a16_status, &zero, sizeof(int));
}

}  // namespace twq
