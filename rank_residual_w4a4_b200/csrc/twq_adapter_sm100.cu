// Low-rank adapters of many requests beside the shared layer, on the 5th-generation
// tensor cores: the three products that the forward and the backward pass consist of,
// each over tiles of at most 128 rows of one adapter (the rows grouped by adapter,
// twq_group.cu), gathered by row number.
//
//   shrink   H = Z W^T       rows x r    forward Z = X, W = A;  backward Z = dY, W = B^T
//   expand   Y = base + s H W^T          forward W = B, H = h;  backward W = A^T, H = dh
//   outer    D_g = sum over rows Z^T H   dB from dY and h;      dA from X and dh
//
// All three are bound by HBM: 2 r operations for each element of X, Y or their gradients
// that is read or written, against some 250 per byte that the tensor cores could do. So
// each streams its large operand once through shared memory and leaves the products to
// tcgen05.mma with fp32 accumulators in tensor memory.
// A tile whose rows follow one another in the batch (a request's prompt) comes by TMA; rows that
// stand anywhere by 16-byte cp.async, into the same 128-byte-swizzle layout. Measured on 8192 rows
// of 25600: TMA tiles 6.0 TB/s, TMA row gathers (4 rows an instruction) 3.8, cp.async 4.8.
// Where rows of a tile are summed, its missing rows are zeros, and ranks beyond r always are,
// so nothing of another row or adapter takes part in a product.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "sm100_ptx.cuh"
#include "twq_adapter.h"

namespace twq {

__device__ int g_adapter_status;

namespace {

// A wait that lasts 2 s is a failure (the kernels' limit: AdapterCall::wait_ns, which is this but in
// the self-test).
constexpr uint64_t kWaitLimitNs = kAdapterWaitNs;
constexpr int kSms = 148;
constexpr int kMaxSmem = 226 * 1024;  // dynamic; the kernels' static part is 1 KB

// Site codes of the bounded waits.
enum : int { kSiteEmpty = 61, kSiteFull, kSiteAccEmpty, kSiteDone, kSiteHEmpty, kSiteDrain, kSiteEnd, kSiteLand };

struct WaitState {  // a block's, in shared memory
  int gave_up;
  uint64_t ns;  // limit of a wait
};
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile WaitState* w, int site) {
  const uint64_t t0 = global_timer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (w->gave_up) return false;
    if (global_timer_ns() - t0 > w->ns) {
      atomicCAS(&g_adapter_status, 0, site);
      w->gave_up = 1;
      return false;
    }
  }
}
// Bounded wait; false once the block is giving up.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile WaitState* w, int site) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, w, site);
}

// The same for a whole warp: one answer for all of its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile WaitState* w, int site) {
  return __all_sync(0xFFFFFFFFu, wait(bar, parity, w, site));
}
// Waits for MMAs in flight, which complete by themselves, on every way out of a kernel (their
// issuer may take kWaitLimitNs to give up its own wait, so twice that).
__device__ __forceinline__ void wait_mmas(uint64_t* bar) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, 0)) {
    if (global_timer_ns() - t0 > 2 * kWaitLimitNs) {
      atomicCAS(&g_adapter_status, 0, kSiteEnd);
      break;
    }
  }
}

// What a block that gives up does about its TMA copies in flight: they must land before it leaves.
// The copies of steps [issued - slots, issued) of a ring may be; every earlier one has been used.
// `missing`: how many of a step's arrivals will not come any more, because their threads gave up
// before it; they are made up for here, so that the step's phase ends once its bytes are there.
__device__ __noinline__ void land(uint64_t* bar, uint32_t parity, int missing) {
  if (missing > 0)
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
                 "r"(missing)
                 : "memory");
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      atomicExch(&g_adapter_status, kSiteLand);
      return;
    }
  }
}
template <typename Missing>
__device__ __forceinline__ void land_ring(uint64_t* full, int slots, int issued, Missing missing) {
  for (int step = max(0, issued - slots); step < issued; ++step)
    land(&full[step % slots], (step / slots) & 1, missing(step));
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
// One arrival on `bar` (whose count includes it) once all cp.async of this thread so far have
// landed. The thread goes on at once, so the depth of the loads is the number of stages, not
// what the loading threads can wait for. The reader of the data fences the proxies. Each
// arrival takes the barrier about 2 cycles (320 of them: 0.35 us a stage, of the 0.7 us that
// a 32 KB stage takes from HBM), so few threads load, with many copies each.
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// The arrivals of a warp by its lane 0, for a barrier that counts the threads of the other way to
// load. Each loading warp makes its own: a warp that only waited, for its turn in the ring, could
// fall two turns behind the one that issues the copies, and then wait for a phase long past.
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(count)
               : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x,
                                         int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}
// The same for what is read once: first to leave L2, which then keeps what is read again (weights,
// H, and the parts that the backward pass adds up).
__device__ __forceinline__ uint64_t read_once_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_once(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x,
                                              int y, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "l"(policy)
      : "memory");
}
// 64 columns of `rows` rows from row y on, in boxes of 128 rows or, for a part of that, of 16: the
// bytes that this will complete, and the copies.
__device__ __forceinline__ uint32_t rows_bytes(int rows) { return (rows + 15) / 16 * 2048; }
template <bool kOnce>
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, const CUtensorMap* map16,
                                              uint64_t* bar, int x, int y, int rows) {
  const uint64_t once = kOnce ? read_once_policy() : 0;
  auto load = [&](uint32_t d, const CUtensorMap* m, int yy) {
    if (kOnce)
      tma_load_once(d, m, bar, x, yy, once);
    else
      tma_load(d, m, bar, x, yy);
  };
  if (rows > 112) {
    load(dst, map, y);
  } else {
    for (int i = 0; i < rows; i += 16) load(dst + i * 128, map16, y + i);
  }
}
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x,
                                          int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Offset of 16-byte chunk c of row `row` in a tile of 128-byte rows, 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(int row, int c) {
  return static_cast<uint32_t>(row * 128 + ((c ^ (row & 7)) << 4));
}

// Shared-memory matrix descriptors (128-byte swizzle) as two words. Low: address / 16 and the
// leading byte offset / 16 (K-major: unused, 1; "MN-major", an operand whose memory rows are the
// reduction index and whose 64-element column blocks lie block_bytes apart: that distance).
// High: 8-row groups 1024 bytes apart, descriptor version 1, swizzle code 2. Steps along the
// reduction add to the low word alone: built anew for each MMA, the descriptors took the one
// issuing thread as long as the MMAs themselves (100 cycles each instead of 60).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// The address is masked to its field: in a cluster, bits above it say which block's memory it is.
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) {
  return ((saddr >> 4) & 0x3FFFu) | (1u << 16);
}
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr, uint32_t block_bytes) {
  return ((saddr >> 4) & 0x3FFFu) | ((block_bytes >> 4) << 16);
}
constexpr uint32_t kAMajorMn = 1u << 15, kBMajorMn = 1u << 16;

// D[tmem] (+)= A B^T, bf16 x bf16 -> fp32.
__device__ __forceinline__ void mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                    bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %4};\n\t"
      "mov.b64 b, {%2, %4};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(kDescHi), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

// The same with A in tensor memory: a lane per row, two elements a column.
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc,
                                           bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %4};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "n"(kDescHi), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 4 int8 codes -> their values times s, rounded to BF16. The code plus 128 becomes the low
// mantissa byte of 2^23, so the subtraction is exact and only the product is rounded. BF16
// is the type that the activation had; an fp32 operand would halve the MMA rate.
__device__ __forceinline__ uint2 dequant4(uint32_t w, uint64_t s2) {
  const uint32_t u = w ^ 0x80808080u;
  const uint64_t bias = f2_pack(-8388736.0f, -8388736.0f);
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t q = f2_pack(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 | (2 * i))),
                               __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 | (2 * i + 1))));
    float lo, hi;
    f2_unpack(f2_mul(f2_add(q, bias), s2), lo, hi);
    o[i] = pack2(lo, hi);
  }
  return make_uint2(o[0], o[1]);
}
__device__ __forceinline__ void dequant16(uint4 q, float scale, uint4& a, uint4& b) {
  const uint64_t s = f2_pack(scale, scale);
  const uint2 p0 = dequant4(q.x, s), p1 = dequant4(q.y, s), p2 = dequant4(q.z, s),
              p3 = dequant4(q.w, s);
  a = make_uint4(p0.x, p0.y, p1.x, p1.y);
  b = make_uint4(p2.x, p2.y, p3.x, p3.y);
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float lds4(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ float4 ld_peer16(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint8_t* align1k(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// Four columns of a row of a BF16 matrix of rank r; split: of rows of 2 r, the values rounded and,
// r columns on, what the rounding left (together 16 bits of the value).
__device__ __forceinline__ void store_value(uint16_t* out, int64_t row, int r, int c, float4 v, bool split) {
  const uint2 hi = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
  if (!split) {
    *reinterpret_cast<uint2*>(out + row * r + c) = hi;
    return;
  }
  *reinterpret_cast<uint2*>(out + row * 2 * r + c) = hi;
  // nothing is left of an infinity (or of what rounds to one)
  auto left = [](float x, float h) { return fabsf(h) <= 3.4e38f ? x - h : 0.0f; };
  *reinterpret_cast<uint2*>(out + row * 2 * r + r + c) =
      make_uint2(pack2(left(v.x, lo_f(hi.x)), left(v.y, hi_f(hi.x))),
                 pack2(left(v.z, lo_f(hi.y)), left(v.w, hi_f(hi.y))));
}

// The sum of the two terms' products. Where X holds an infinity the first term alone has the sign:
// the second, which may be zero or of the other sign, would make a NaN of it.
__device__ __forceinline__ float both_terms(float v, float w) { return isfinite(v) ? v + w : v; }

// A block's work items, each a part of a row tile: item k is number first + stride k, in tile
// number / parts.
struct Items {
  int first, stride, parts, count;
  __device__ __forceinline__ int tile(int k) const { return (first + stride * k) / parts; }
};

// The rows of each item's tile that one thread loads (row `first` + step j of the tile; -1
// beyond its end), known an item ahead, and the tile itself two ahead, so that no load of
// Z, base or H waits for a look-up.
template <int kRows>
struct RowsAhead {
  const int4* tiles;
  const int32_t* order;
  Items items;
  int at, first, step;
  int row[kRows], next[kRows];
  int group, next_group;
  int run, next_run;    // first row of a tile whose rows follow one another, else -1
  int count, next_count;
  int4 after;

  __device__ __forceinline__ int4 load_tile(int k) const {
    return k < items.count ? __ldg(tiles + items.tile(k)) : make_int4(-1, 0, 0, -1);
  }
  __device__ __forceinline__ void look_up(const int4& t, int (&r)[kRows]) const {
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int i = first + step * j;
      r[j] = i < t.z ? __ldg(order + t.y + i) : -1;
    }
  }
  __device__ __forceinline__ void start(const int4* tl, const int32_t* ord, const Items& it, int f, int st) {
    tiles = tl, order = ord, items = it, at = 0, first = f, step = st;
    const int4 t0 = load_tile(0), t1 = load_tile(1);
    after = load_tile(2);
    look_up(t0, row);
    look_up(t1, next);
    group = t0.x, next_group = t1.x;
    run = t0.w, next_run = t1.w;
    count = t0.z, next_count = t1.z;
  }
  __device__ __forceinline__ void advance() {
    ++at;
#pragma unroll
    for (int j = 0; j < kRows; ++j) row[j] = next[j];
    group = next_group, run = next_run, count = next_count;
    look_up(after, next);
    next_group = after.x, next_run = after.w, next_count = after.z;
    after = load_tile(at + 2);
  }
};

// ------------------------------------------------------------------ shrink
struct ShrinkArgs {
  CUtensorMap map, map16;  // Z: 128 or 16 rows x 64 columns; with codes, map: 32 rows x 64 pairs
  CUtensorMap wmap;  // W: rp rows x 64 of k, or (kTrans) 64 rows of k x 64 of r
  const int4* tiles;
  const int32_t* order;
  int cap16;
  const uint16_t* z;  // BF16 rows (stride ldz), or codes
  int64_t ldz;
  const int8_t* q;
  const float* sq;
  const float* scale; // or null: 1
  uint16_t* out;      // b x r, or (split) b x 2 r: the value in BF16, and what that leaves
  int k, r, rp;       // rp: r rounded up to 16
  bool split;
  // Tiles of Z, 128 x 64, each with its W; with codes: groups of a team, groups of W.
  int stages, wstages;
  uint64_t wait_ns;
  int stall;          // self-test: the copies of Z end half way (codes: they are not used)
};

constexpr int kShrinkThreads = 320;  // 8 warps load Z, then epilogue; MMA warp; TMA warp
constexpr int kShrinkStages = 8;     // at most, of either kind
constexpr uint32_t kShrinkTmemCols = 128;  // and as many for two groups of converted codes
// Codes are converted by two teams of four warps, which take the groups of 128 columns in turn. A
// warp has 32 rows, for which it keeps its own ring of raw codes (TMA where the rows follow one
// another), a lane a row, and leaves the BF16 in tensor memory, where the MMA takes A from: no
// proxy fence and no second turn through shared memory. 4096 x 14336, rank 16: 28 us, against 31
// with all eight warps on each group and A in shared memory. Of the 28 us the eight groups of a team
// are 13 (1.6 a group, 1.2 of it conversion while four teams share the SM's integer pipe); the rest
// is the start, the first copies and the joining of the parts. The conversion of all codes, seven
// operations at half rate for four, would take that pipe 5.7 us. A team has one buffer in tensor
// memory, so it waits for the products of its last group before it writes the next.

// One row tile per cluster, whose blocks split the reduction over k (block `rank` takes the groups
// of 128 columns rank, rank + splits, ..., so that they read neighbouring pieces of the rows at
// about the same time) and add their parts through distributed shared memory in rank order.
// Bound by the copies of Z, and by the start and the joining of the parts (some 6 us) where Z is
// small: 8192 x 5120, rank 64: 24 us, 3.6 TB/s; 2048 x 4096, rank 32: 12 us.
template <bool kCodes, bool kTrans>
__global__ void __launch_bounds__(kShrinkThreads, 2)
    shrink_kernel(const __grid_constant__ ShrinkArgs p) {
  // A step: 64 columns, or a group of 128 with codes.
  constexpr int kPer = kCodes ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_full[kShrinkStages], s_empty[kShrinkStages], s_wfull[kShrinkStages],
      s_wempty[kShrinkStages], s_raw[kCodes ? 16 : 1], s_done;
  __shared__ uint32_t s_tmem;
  __shared__ WaitState s_wait;
  __shared__ int s_steps[8], s_issued;  // of each loading warp; of the TMA
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int splits = gridDim.x, rank = blockIdx.x;  // the cluster spans the grid's x
  if (tid == 288) {
    tma_prefetch_desc(&p.map);
    tma_prefetch_desc(&p.wmap);
  }
  pdl_launch_dependents();
  pdl_wait();
  const int number = p.tiles[0].y;
  const int4 t = p.tiles[1 + p.cap16 + blockIdx.y];  // written or not, it is in the list's room
  if (static_cast<int>(blockIdx.y) >= number) return;
  if (t.x < 0) {  // rows without adapter
    for (int i = rank * kShrinkThreads + tid; i < t.z * (p.r / 8); i += splits * kShrinkThreads) {
      const int64_t row = p.order[t.y + i / (p.r / 8)];
      if (!p.split) *reinterpret_cast<uint4*>(p.out + row * p.r + i % (p.r / 8) * 8) = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  uint8_t* smem = align1k(smem_raw);
  const uint32_t sz = smem_u32(smem);
  const uint32_t sw = sz + p.stages * kPer * 16384;  // with codes: two teams' groups of 16 KB
  const int wbytes = kTrans ? (p.rp + 63) / 64 * 8192 : p.rp * 128;
  // rows beyond a partial tile's end then hold anything; their sums are not stored
  const bool tma = t.w >= 0;
  const int groups = (p.k / 128 - rank + splits - 1) / splits;
  const int steps = groups * 2 / kPer;
  const int z_steps = p.stall ? steps / 2 : steps;
  const int tma_steps = !kCodes && tma ? z_steps : steps;
  auto column = [&](int tile) { return (rank + (tile >> 1) * splits) * 128 + (tile & 1) * 64; };
  // W's part of a step. Without kTrans the rows beyond r are the next adapter's (or zeros): they
  // only reach accumulator columns that are not stored.
  auto load_w = [&](int step, int slot, uint64_t* bar) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t dst = sw + (slot * kPer + i) * wbytes;
      if constexpr (kTrans) {
        tma_load3(dst, &p.wmap, bar, 0, column(step * kPer + i), t.x);
        if (p.rp > 64) tma_load3(dst + 8192, &p.wmap, bar, 64, column(step * kPer + i), t.x);
      } else {
        tma_load(dst, &p.wmap, bar, column(step * kPer + i), t.x * p.r);
      }
    }
  };
  auto load_both = [&](int step, int slot) {
    mbar_arrive_expect_tx(&s_full[slot], (tma ? rows_bytes(t.z) : 0) + wbytes);
    if (tma) tma_load_rows<true>(sz + slot * 16384, &p.map, &p.map16, &s_full[slot], column(step), t.w, t.z);
    load_w(step, slot, &s_full[slot]);
  };
  if (tid == 288) {
    // codes: a team's four warps, and W's own barriers; else the loading threads and the TMA
    for (int i = 0; i < (kCodes ? 2 : p.stages); ++i) {
      mbar_init(&s_full[i], kCodes ? 4 : tma ? 1 : 257);
      mbar_init(&s_empty[i], 1);
    }
    for (int i = 0; kCodes && i < p.wstages; ++i) {
      mbar_init(&s_wfull[i], 1);
      mbar_init(&s_wempty[i], 1);
    }
    for (int i = 0; kCodes && i < 16; ++i) mbar_init(&s_raw[i], 1);
    mbar_init(&s_done, 1);
    s_wait.gave_up = 0;
    s_wait.ns = p.wait_ns;
    fence_barrier_init();
    s_issued = min(tma_steps, kCodes ? p.wstages : p.stages);
    for (int step = 0; step < s_issued; ++step) {
      if (kCodes) {
        mbar_arrive_expect_tx(&s_wfull[step], kPer * wbytes);
        load_w(step, step, &s_wfull[step]);
      } else {
        load_both(step, step);
      }
    }
  }
  constexpr uint32_t kCols = kShrinkTmemCols * (kCodes ? 2 : 1);
  if (warp == 8) {
    tmem_alloc(&s_tmem, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  if (warp == 9) {
    if (lane == 0) {
      const int ring = kCodes ? p.wstages : p.stages;
      int slot = 0, step = s_issued;
      uint32_t phase = 0;
      for (; step < tma_steps; ++step) {
        if (!wait(kCodes ? &s_wempty[slot] : &s_empty[slot], phase, &s_wait, kSiteEmpty)) break;
        if (kCodes) {
          mbar_arrive_expect_tx(&s_wfull[slot], kPer * wbytes);
          load_w(step, slot, &s_wfull[slot]);
        } else {
          load_both(step, slot);
        }
        if (++slot == ring) {
          slot = 0;
          phase ^= 1u;
        }
      }
      s_issued = step;
    }
  } else if (kCodes && warp < 8) {
    if constexpr (kCodes) {
      const int team = warp >> 2, sub = warp & 3;
      const bool any = sub * 32 < t.z;  // else this warp has no row
      const int mine = (groups + 1 - team) / 2;  // groups team, team + 2, ...
      const int row = sub * 32 + lane < t.z ? __ldg(p.order + t.y + sub * 32 + lane) : -1;
      const int two = p.stages - 1;  // 1 or 2 groups in the ring
      const uint32_t raw = sz + warp * p.stages * 4096;
      const uint64_t once = read_once_policy();
      auto fetch = [&](int j) {
        if (any && j < mine) {
          const int col = (rank + (team + 2 * j) * splits) * 128;
          const uint32_t dst = raw + (j & two) * 4096;
          if (tma) {
            if (lane == 0) {
              uint64_t* bar = &s_raw[warp * 2 + (j & two)];
              mbar_arrive_expect_tx(bar, 4096);
              tma_load_once(dst, &p.map, bar, col / 2, t.w + sub * 32, once);
            }
          } else {
            const int ch = lane & 7;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = 4 * i + (lane >> 3);
              const int from = __shfl_sync(0xffffffffu, row, rr);
              cp16(dst + sw128(rr, ch), p.q + static_cast<int64_t>(max(from, 0)) * p.k + col + ch * 16,
                   from >= 0);
            }
          }
        }
        if (!tma) cp_commit();
      };
      for (int j = 0; j <= two; ++j) fetch(j);
      // Scales of three groups, each loaded into its own register three groups ahead (a move
      // between registers would wait for the load).
      const float* scales = p.sq + static_cast<int64_t>(max(row, 0)) * (p.k >> 7) + rank + team * splits;
      auto scale_of = [&](int j) { return row >= 0 && j < mine ? __ldg(scales + j * 2 * splits) : 0.0f; };
      float sc[3];
#pragma unroll
      for (int u = 0; u < 3; ++u) sc[u] = scale_of(u);
      const uint32_t ta = tmem + (static_cast<uint32_t>(sub * 32) << 16) + kShrinkTmemCols + team * 64;
      bool alive = !p.stall;
      int asked = two + 1;  // groups that fetch was called for
      for (int base = 0; base < mine && alive; base += 3) {
#pragma unroll
        for (int u = 0; u < 3; ++u) {
          const int j = base + u;
          if (j >= mine || !alive) break;
          uint4 v[8];
          if (any) {
            if (tma) {
              alive = warp_wait(&s_raw[warp * 2 + (j & two)], (j >> two) & 1, &s_wait, kSiteFull);
            } else if (two) {
              cp_wait<1>();
            } else {
              cp_wait<0>();
            }
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = lds16(raw + (j & two) * 4096 + sw128(lane, q));
          }
          alive = alive && (j == 0 || warp_wait(&s_empty[team], (j - 1) & 1, &s_wait, kSiteEmpty));
          if (!alive) break;
          if (any) {
            tc_fence_after();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t o[32];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint4 a, b;
                dequant16(v[half * 4 + q], sc[u], a, b);
                o[q * 8] = a.x, o[q * 8 + 1] = a.y, o[q * 8 + 2] = a.z, o[q * 8 + 3] = a.w;
                o[q * 8 + 4] = b.x, o[q * 8 + 5] = b.y, o[q * 8 + 6] = b.z, o[q * 8 + 7] = b.w;
              }
              tmem_st32(ta + half * 32, o);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(&s_full[team]);
          // Only here have all lanes' reads of the slot surely ended: their values are in tensor
          // memory. (Requested right behind the loads of v, new codes reached some lanes instead
          // of the old ones when this warp then waited for the MMAs.)
          fetch(j + 1 + two);
          asked = j + 2 + two;
          sc[u] = scale_of(j + 3);
        }
      }
      if (!alive && any && tma && lane == 0)
        for (int j = max(0, asked - 1 - two); j < min(asked, mine); ++j)
          land(&s_raw[warp * 2 + (j & two)], (j >> two) & 1, 0);
      cp_wait_all();
    }
  } else if (warp < 8 && !tma) {
    // Thread: rows tid / 8 + 32 j, chunk tid % 8.
    const int r0 = tid >> 3, ch = tid & 7;
    int row[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) row[j] = r0 + j * 32 < t.z ? __ldg(p.order + t.y + r0 + j * 32) : -1;
    int slot = 0, step = 0;
    uint32_t phase = 0;
    for (; step < z_steps; ++step) {
      if (step >= p.stages && !warp_wait(&s_empty[slot], phase ^ 1u, &s_wait, kSiteEmpty)) break;
      const uint32_t zs = sz + slot * 16384;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        cp16(zs + sw128(r0 + j * 32, ch), p.z + max(row[j], 0) * p.ldz + column(step) + ch * 8,
             row[j] >= 0);
      cp_arrive(&s_full[slot]);
      if (++slot == p.stages) {
        slot = 0;
        phase ^= 1u;
      }
    }
    if (lane == 0) s_steps[warp] = step;
    cp_wait_all();
  } else if (warp == 8 && lane == 0) {
    const uint32_t idesc = idesc_bf16(p.rp) | (kTrans ? kBMajorMn : 0u);
    int slot = 0, wslot = 0;  // with codes, slot: the team whose group it is
    uint32_t phase = 0, wphase = 0;
    for (int step = 0; step < steps; ++step) {
      if (kCodes && !wait(&s_wfull[wslot], wphase, &s_wait, kSiteFull)) break;
      if (!wait(&s_full[slot], phase, &s_wait, kSiteFull)) break;
      if (!kCodes && !tma) fence_proxy_async_smem();
      tc_fence_after();
      if constexpr (kCodes) {
        const uint32_t a = tmem + kShrinkTmemCols + slot * 64, b = desc_k(sw + wslot * 2 * wbytes);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_tmem_a(tmem, a + k * 8, b + (k >> 2) * (wbytes >> 4) + (k & 3) * 2, idesc, step + k > 0);
        mma_commit(&s_wempty[wslot]);
        if (++wslot == p.wstages) {
          wslot = 0;
          wphase ^= 1u;
        }
      } else {
        const uint32_t a = desc_k(sz + slot * 16384), ws = sw + slot * wbytes;
        const uint32_t b = kTrans ? desc_mn(ws, 8192) : desc_k(ws);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma(tmem, a + k * 2, b + k * (kTrans ? 128 : 2), idesc, step + k > 0);
      }
      mma_commit(&s_empty[slot]);
      if (++slot == (kCodes ? 2 : p.stages)) {
        slot = 0;
        phase ^= 1u;
      }
    }
    mma_commit(&s_done);
  }
  __syncwarp();

  // Parts to shared memory (the stages are free once every MMA has completed), then each
  // block of the cluster adds a share of the rows over the blocks.
  float* part = reinterpret_cast<float*>(smem);
  const int pitch = p.rp + 4;
  const int lo = rank * 128 / splits, hi = min(t.z, (rank + 1) * 128 / splits);
  const int quads = p.r / 4;
  const float f = p.scale ? p.scale[t.x] : 1.0f;
  const int row0 = lo + tid / quads < hi ? p.order[t.y + lo + tid / quads] : 0;
  wait_mmas(&s_done);
  __syncwarp();
  if (warp < 8) {
    tc_fence_after();
    const int i = (warp & 3) * 32 + lane;
    for (int c = (warp >> 2) * 8; c < p.rp; c += 16) {
      uint32_t v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (steps > 0) {
        tmem_ld8(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c, v);
        tmem_wait_ld();
      }
#pragma unroll
      for (int u = 0; u < 8; u += 4)
        *reinterpret_cast<uint4*>(part + i * pitch + c + u) =
            make_uint4(v[u], v[u + 1], v[u + 2], v[u + 3]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (s_wait.gave_up && tid == 288) {
    if constexpr (kCodes) {
      land_ring(s_wfull, p.wstages, s_issued, [](int) { return 0; });
    } else {
      land_ring(s_full, p.stages, s_issued, [&](int step) {
        int missing = 0;
        for (int w = 0; !tma && w < 8; ++w) missing += s_steps[w] <= step ? 32 : 0;
        return missing;
      });
    }
  }
  __syncwarp();
  if (warp == 8) tmem_dealloc(tmem, kCols);
  if (splits > 1) cluster_sync_startup();
  for (int i = tid; i < (hi - lo) * quads; i += kShrinkThreads) {
    const int rr = lo + i / quads, c = i % quads * 4;
    const uint32_t at = smem_u32(part + rr * pitch + c);
    float4 o[8];
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s < splits) o[s] = ld_peer16(map_peer(at, s));
    float4 v = o[0];
#pragma unroll
    for (int s = 1; s < 8; ++s)
      if (s < splits) v.x += o[s].x, v.y += o[s].y, v.z += o[s].z, v.w += o[s].w;
    const int64_t orow = i == tid ? row0 : p.order[t.y + rr];
    store_value(p.out, orow, p.r, c, make_float4(v.x * f, v.y * f, v.z * f, v.w * f), p.split);
  }
  if (splits > 1) cluster_sync_startup();  // peers may still be reading this block's part
}

// --------------------------------------------------------------------- sum
__host__ __device__ __forceinline__ int chunk_begin(int c, int chunks, int tiles) {
  return static_cast<int>(static_cast<int64_t>(c) * tiles / chunks);
}

// What the outer products leave to be added up: dh from its slices' parts, and the groups of dA and
// dB that the chunks cut. Right after the kernel that wrote them, while the parts are in L2 (at the
// end of the call those of dY were not: 18 us instead of 11 at 8192 x 5120 x 25600).
struct SumArgs {
  const int4* tiles;
  const int32_t *order, *offsets, *first128;
  int b, count, r;
  // dh, as rows of 2 r (store_value), from slices x r / 4 x b x 4
  const float* dpart;
  uint16_t* dh;
  int slices, dh_blocks;
  // parts [block][rank / 4][column of the block][4]; out count x r x k (dA) or count x k x r (dB)
  struct {
    const float* part;
    uint16_t* out;
    int k, chunks, blocks;  // blocks of threads for each group
  } side[2];
};

// Largest c with chunk_begin(c) <= tile.
__device__ __forceinline__ int chunk_of(int tile, int chunks, int tiles) {
  int c = static_cast<int>(static_cast<int64_t>(tile) * chunks / tiles);
  while (chunk_begin(c + 1, chunks, tiles) <= tile) ++c;
  return c;
}

// A thread: 4 ranks of a position; slices in order.
__device__ __forceinline__ void sum_dh(const SumArgs& p, int block) {
  const int wide = (p.b + 255) / 256, quad = block / wide;
  const int64_t pos = static_cast<int64_t>(block - quad * wide) * 256 + threadIdx.x;
  if (pos >= p.offsets[p.count]) return;
  const int64_t row = p.order[pos], step = static_cast<int64_t>(p.b) * p.r;
  const float* part = p.dpart + (static_cast<int64_t>(quad) * p.b + pos) * 4;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int s = 0; s < p.slices; ++s) {
    const float4 o = __ldcg(reinterpret_cast<const float4*>(part + s * step));
    v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
  }
  store_value(p.dh, row, p.r, quad * 4, v, true);
}

// A thread: 8 ranks of a column of group g; chunks in order. Zeros for a group without rows.
template <bool kByRank>
__device__ __forceinline__ void sum_group(const SumArgs& p, int block) {
  const auto& side = p.side[kByRank ? 0 : 1];
  const int g = block / side.blocks, oct = p.r / 8;
  const int64_t i = static_cast<int64_t>(block - g * side.blocks) * 256 + threadIdx.x;
  const int64_t blk = i / (oct * 128);
  if (blk >= side.k / 128) return;
  const int rest = static_cast<int>(i - blk * (oct * 128));
  const int c = rest / 128 * 8, j = static_cast<int>(blk) * 128 + rest % 128;
  const int gb = p.first128[g], ge = p.first128[g + 1], total = p.first128[p.count];
  const int64_t size = static_cast<int64_t>(side.k) * p.r;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f), w = v;
  if (gb < ge) {
    const int chunks = min(side.chunks, total);
    const int c0 = chunk_of(gb, chunks, total), c1 = chunk_of(ge - 1, chunks, total);
    if (c0 == c1) return;  // inside one chunk: already written
    // the group's run is a chunk's second one only where the group starts inside it
    const float* part = side.part + (blk * (p.r / 4) + c / 4) * 512 + rest % 128 * 4;
    const float* first = part + (2 * c0 + (gb > chunk_begin(c0, chunks, total) ? 1 : 0)) * size;
    v = __ldcg(reinterpret_cast<const float4*>(first));
    w = __ldcg(reinterpret_cast<const float4*>(first + 512));
#pragma unroll 4
    for (int x = c0 + 1; x <= c1; ++x) {
      const float4 a = __ldcg(reinterpret_cast<const float4*>(part + 2 * x * size));
      const float4 b = __ldcg(reinterpret_cast<const float4*>(part + 2 * x * size + 512));
      v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
      w.x += b.x, w.y += b.y, w.z += b.z, w.w += b.w;
    }
  }
  const uint32_t o[4] = {pack2(v.x, v.y), pack2(v.z, v.w), pack2(w.x, w.y), pack2(w.z, w.w)};
  uint16_t* out = side.out + g * size;
  if (kByRank) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      out[static_cast<int64_t>(c + 2 * e) * side.k + j] = static_cast<uint16_t>(o[e]);
      out[static_cast<int64_t>(c + 2 * e + 1) * side.k + j] = static_cast<uint16_t>(o[e] >> 16);
    }
  } else {
    *reinterpret_cast<uint4*>(out + static_cast<int64_t>(j) * p.r + c) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

__device__ __forceinline__ void sum_block(const SumArgs& p, int block) {
  if (block < p.dh_blocks) return sum_dh(p, block);
  block -= p.dh_blocks;
  if (block < p.side[0].blocks * p.count) return sum_group<true>(p, block);
  sum_group<false>(p, block - p.side[0].blocks * p.count);
}

__global__ void __launch_bounds__(256) sum_kernel(const SumArgs p) {
  pdl_launch_dependents();
  pdl_wait();
  sum_block(p, blockIdx.x);
}

// ------------------------------------------------------------------ expand
struct ExpandArgs {
  CUtensorMap map, map16;  // base: 128 or 16 rows x 64 columns
  CUtensorMap hmap;  // H: 128 rows x 64 of r
  CUtensorMap wmap;  // W: 64 columns x 64 of r, or (kTrans) rp of r x 64 columns
  const int4* tiles;
  const int32_t* order;
  int cap16;
  const uint16_t* h;  // b rows of r, ldh apart
  const float* scale; // or null: 1
  const uint16_t* base;
  uint16_t* y;
  const int32_t *first128, *offsets;
  int b, count;
  int n, r, rp, ldh;
  int stage_bytes, slots, hslots, bslots;  // a W stage; W stages; H tiles; base stages of 16 KB
  int segs;
  SumArgs sum;  // kSums: what the kernel in front left to be added up, `sums` blocks of 256 threads
  int sums;
  uint64_t wait_ns;
  int stall;    // self-test: one of the two loading warps stops at the first unit
};

constexpr int kExpandThreads = 384;  // 8 epilogue warps; MMA; 2 warps load H and base; TMA of W
// At most. The two halves of the epilogue warps take turns, so both numbers are even: a slot then
// belongs to one half, and its barrier is never a whole turn ahead of a waiter.
constexpr int kExpandSlots = 4;      // W stages, and accumulators of 64 columns
constexpr int kBaseSlots = 4;        // base stages
constexpr int kExpandBars = 256;     // bytes behind the base stages: barriers, what goes with them

__device__ __forceinline__ uint4 ld_stream(const void* ptr) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(ptr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_stream(void* ptr, uint4 v) {
  asm volatile("st.global.L1::no_allocate.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(ptr), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// Items: `segs` parts of each tile with an adapter, of about 8 units of 64 columns; the grid's
// blocks take them in turn, so that at any time they work on neighbouring columns of a few row
// tiles (a copy by blocks with a long part of a row tile each: 4.6 TB/s; with short ones in
// turn: 5.8). base comes through shared memory, several stages ahead. A lane of the epilogue takes
// a row: it adds its accumulators to the row's base in the stage, in place, and its warp copies the
// stage out, 128 bytes of a row at a time; base may be y itself: an element is written after the
// only read of it. Measured, whole calls of 8192 x 5120 x 25600, rank 64: 174 us, of which this
// kernel is some 150 (842 MB, 5.6 TB/s; a copy of as much takes 129). With the hint that base is
// read once, which the other kernels gain by: 186 (with four sets of buffers in turn, base apart
// from y, the other way round: 188, and 181 with it). Slower when they were tried: stages sent out
// by TMA, free later (191); accumulators read in the 16x256b form and stores from registers, 1.5
// times the instructions (by 10 us, and for 5120 columns of W^T 43 instead of 39).
// dx is made from dh's first term alone: with both, a tile of H would take 16 KB more at rank 64,
// the room of two stages of W.
// Launched so that it may start before the kernel that writes H has ended: until then it reads
// only what that kernel does not write (the grouping, W, base) and writes nothing.
template <bool kTrans, bool kSums>
__global__ void __launch_bounds__(kExpandThreads, 2) expand_kernel(const __grid_constant__ ExpandArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];  // no other shared memory: two blocks fill an SM
  const int kt = (p.rp + 63) / 64;  // 64-wide tiles of the reduction
  const uint32_t sh = smem_u32(smem);
  const uint32_t sw = sh + p.hslots * kt * 16384;
  const uint32_t sb = sw + p.slots * p.stage_bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (sb - sh) + p.bslots * 16384);
  uint64_t* s_full = bars;                          // W stage
  uint64_t* s_done = s_full + kExpandSlots;         // accumulator (and its W stage read)
  uint64_t* s_free = s_done + kExpandSlots;
  uint64_t* s_bfull = s_free + kExpandSlots;
  uint64_t* s_bfree = s_bfull + kBaseSlots;
  uint64_t* s_hfull = s_bfree + kBaseSlots;
  uint64_t* s_hfree = s_hfull + 2;
  uint64_t* s_end = s_hfree + 2;
  WaitState* s_wait = reinterpret_cast<WaitState*>(s_end + 1);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_wait + 1);
  int* s_units = reinterpret_cast<int*>(s_tmem + 1);  // what each loading warp has asked for: base,
  int* s_items = s_units + 2;                         // H,
  int* s_w = s_items + 2;                             // W
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int units = p.n / 64;
  const int total = p.first128[p.count] * p.segs;
  Items items{static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), p.segs, 0};
  items.count = (total - items.first + items.stride - 1) / items.stride;  // <= 0: none
  const int4* tiles = p.tiles + 1 + p.cap16;
  // units of item k
  auto unit_begin = [&](int k) { return (items.first + items.stride * k) % p.segs * units / p.segs; };
  auto unit_end = [&](int k) { return ((items.first + items.stride * k) % p.segs + 1) * units / p.segs; };

  auto add_up = [&]() {  // by warps 0 .. 7, while the first copies are under way
    if (!kSums) return;
    pdl_wait();
    for (int i = blockIdx.x; i < p.sums; i += gridDim.x) sum_block(p.sum, i);
  };
  if (items.count <= 0) {
    if (warp < 8) add_up();
  } else {
    if (tid == 0) {
      for (int i = 0; i < kExpandSlots; ++i) {
        mbar_init(&s_full[i], 1);
        mbar_init(&s_done[i], 1);
        mbar_init(&s_free[i], 4);
      }
      for (int i = 0; i < kBaseSlots; ++i) {
        mbar_init(&s_bfull[i], 64);
        mbar_init(&s_bfree[i], 4);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&s_hfull[i], 64);
        mbar_init(&s_hfree[i], 1);
      }
      mbar_init(s_end, 1);
      s_wait->gave_up = 0;
      s_wait->ns = p.wait_ns;
      fence_barrier_init();
    }
    if (warp == 8) {
      tmem_alloc(s_tmem, 64 * kExpandSlots);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp < 8) {
      // Warps 0 .. 3 take the even units of this block, 4 .. 7 the odd ones, each 32 rows of all 64
      // columns: a warp's chain of waits and loads (about 2000 cycles) then spans two units.
      add_up();
      const int sub = warp & 3, rr = sub * 32 + lane;
      RowsAhead<1> ra;
      ra.start(tiles, p.order, items, rr, 0);
      int turn = warp >> 2;  // 0: the next unit is this warp's
      int slot = 0, bs = 0;
      uint32_t ph = 0, bph = 0;
      bool alive = true;
      for (int k = 0; k < items.count && alive; ++k) {
        const float f = p.scale ? p.scale[ra.group] : 1.0f;
        const uint64_t f2 = f2_pack(f, f);
        const int ue = unit_end(k);
        for (int u = unit_begin(k); u < ue; ++u) {
          if (turn == 0) {
            alive = warp_wait(&s_done[slot], ph, s_wait, kSiteDone) &&
                    warp_wait(&s_bfull[bs], bph, s_wait, kSiteFull);
            if (!alive) break;
            tc_fence_after();
            const uint32_t stage = sb + bs * 16384;
            if (sub * 32 < ra.count) {  // else no row of the tile among this warp's 32
              const uint32_t ta = tmem + (static_cast<uint32_t>(sub * 32) << 16) + slot * 64;
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint32_t v[32];
                tmem_ld32(ta + half * 32, v);
                tmem_wait_ld();
                if (half == 1) {
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) mbar_arrive(&s_free[slot]);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const uint32_t at = stage + sw128(rr, half * 4 + q);
                  const uint4 b = p.base ? lds16(at) : make_uint4(0, 0, 0, 0);
                  const uint32_t bb[4] = {b.x, b.y, b.z, b.w};
                  uint32_t o[4];
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    float lo, hi;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(v[q * 8 + 2 * j]),
                                             __uint_as_float(v[q * 8 + 2 * j + 1])),
                                     f2, f2_pack(lo_f(bb[j]), hi_f(bb[j]))),
                              lo, hi);
                    o[j] = pack2(lo, hi);
                  }
                  sts16(at, make_uint4(o[0], o[1], o[2], o[3]));
                }
              }
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int from = (lane >> 3) + 4 * i;
                const int row = __shfl_sync(0xffffffffu, ra.row[0], from);
                if (row >= 0)
                  st_stream(p.y + static_cast<int64_t>(row) * p.n + u * 64 + (lane & 7) * 8,
                            lds16(stage + sw128(sub * 32 + from, lane & 7)));
              }
            } else if (lane == 0) {
              mbar_arrive(&s_free[slot]);
            }
            // The next copy into this stage may be TMA's, which the barrier alone does not order
            // behind the stores above (nor behind the cp.async that filled the stage).
            if (p.base) fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_bfree[bs]);
          }
          turn ^= 1;
          if (++slot == p.slots) {
            slot = 0;
            ph ^= 1u;
          }
          if (++bs == p.bslots) {
            bs = 0;
            bph ^= 1u;
          }
        }
        ra.advance();
      }
    } else if (warp == 8) {
      if (lane == 0) {
        const uint32_t idesc = idesc_bf16(64) | (kTrans ? kBMajorMn : 0u);
        int slot = 0, hs = 0, i = 0;
        uint32_t ph = 0, hph = 0;
        bool alive = true;
        for (int k = 0; k < items.count && alive; ++k) {
          if (!wait(&s_hfull[hs], hph, s_wait, kSiteFull)) break;
          fence_proxy_async_smem();  // H may have come by cp.async
          const uint32_t hb = desc_k(sh + hs * kt * 16384);
          const int ue = unit_end(k);
          for (int u = unit_begin(k); u < ue; ++u, ++i) {
            alive = wait(&s_full[slot], ph, s_wait, kSiteFull) &&
                    (i < p.slots || wait(&s_free[slot], ph ^ 1u, s_wait, kSiteAccEmpty));
            if (!alive) break;
            tc_fence_after();
            const uint32_t ws = sw + slot * p.stage_bytes, d = tmem + slot * 64;
            const uint32_t b = kTrans ? desc_mn(ws, 0) : desc_k(ws);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (q * 16 < p.rp)
                mma(d, hb + (q >> 2) * 1024 + (q & 3) * 2,
                    b + (kTrans ? q * 128 : (q >> 2) * 512 + (q & 3) * 2), idesc, q > 0);
            mma_commit(&s_done[slot]);
            if (++slot == p.slots) {
              slot = 0;
              ph ^= 1u;
            }
          }
          mma_commit(&s_hfree[hs]);
          if (++hs == p.hslots) {
            hs = 0;
            hph ^= 1u;
          }
        }
        mma_commit(s_end);
        wait_mmas(s_end);
      }
    } else {
      const int chunks = p.rp / 8;
      bool alive = true;
      if (warp < 11) {
        const int r0 = (tid - 288) >> 3, ch = tid & 7;  // rows r0 + 8 j, chunk ch
        RowsAhead<16> ra;
        ra.start(tiles, p.order, items, r0, 8);
        int hs = 0, bs = 0, i = 0;
        uint32_t hph = 0, bph = 0;
        auto load_base = [&](int u) {
          if (!p.base) {
            if (lane == 0) mbar_arrive_n(&s_bfull[bs], 32);
          } else if (ra.run >= 0) {
            if (tid == 288) {
              mbar_arrive_expect_tx(&s_bfull[bs], rows_bytes(ra.count));
              tma_load_rows<false>(sb + bs * 16384, &p.map, &p.map16, &s_bfull[bs], u * 64, ra.run, ra.count);
            }
            if (lane == 0) mbar_arrive_n(&s_bfull[bs], tid == 288 ? 31 : 32);
          } else {
            const uint16_t* src = p.base + u * 64 + ch * 8;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              cp16(sb + bs * 16384 + sw128(r0 + 8 * j, ch),
                   src + static_cast<int64_t>(max(ra.row[j], 0)) * p.n, ra.row[j] >= 0);
            cp_arrive(&s_bfull[bs]);
          }
          if (++bs == p.bslots) {
            bs = 0;
            bph ^= 1u;
          }
        };
        // The first stages of base, then H. Not in the forward pass, where they take HBM from the
        // kernel in front (1500 rows of 4096 x 4096, rank 32: 20.8 us instead of 17.7).
        const int early = kTrans ? min(p.bslots, unit_end(0) - unit_begin(0)) : 0;
        for (; i < early; ++i) load_base(unit_begin(0) + i);
        pdl_wait();
        int loaded = 0;  // tiles of H
        for (int k = 0; k < items.count && alive; ++k) {
          if (k >= p.hslots && !warp_wait(&s_hfree[hs], hph ^ 1u, s_wait, kSiteHEmpty)) break;
          if (ra.run >= 0) {  // rows beyond a partial tile's end are read and not used
            if (tid == 288) {
              mbar_arrive_expect_tx(&s_hfull[hs], kt * 16384);
              for (int c = 0; c < kt; ++c)
                tma_load(sh + (hs * kt + c) * 16384, &p.hmap, &s_hfull[hs], c * 64, ra.run);
            }
            if (lane == 0) mbar_arrive_n(&s_hfull[hs], tid == 288 ? 31 : 32);
          } else {
            for (int c = ch; c < chunks; c += 8)
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const bool in = ra.row[j] >= 0 && c * 8 < p.r;
                cp16(sh + (hs * kt + (c >> 3)) * 16384 + sw128(r0 + 8 * j, ch),
                     p.h + (in ? static_cast<int64_t>(ra.row[j]) * p.ldh + c * 8 : 0), in);
              }
            cp_arrive(&s_hfull[hs]);
          }
          if (++hs == p.hslots) {
            hs = 0;
            hph ^= 1u;
          }
          ++loaded;
          const int ue = unit_end(k);
          for (int u = unit_begin(k) + (k == 0 ? early : 0); u < ue; ++u, ++i) {
            if ((i >= p.bslots && !warp_wait(&s_bfree[bs], bph ^ 1u, s_wait, kSiteEmpty)) ||
                (p.stall && warp == 10)) {
              alive = false;
              break;
            }
            load_base(u);
          }
          ra.advance();
        }
        if (lane == 0) s_units[warp - 9] = i, s_items[warp - 9] = loaded;
      } else {
        if (lane == 0) {
          int slot = 0, i = 0, next = __ldg(&tiles[items.tile(0)].x);
          uint32_t ph = 0;
          for (int k = 0; k < items.count && alive; ++k) {
            const int g = next;
            if (k + 1 < items.count) next = __ldg(&tiles[items.tile(k + 1)].x);
            const int ue = unit_end(k);
            for (int u = unit_begin(k); u < ue; ++u, ++i) {
              // the MMAs that read this stage are done when their accumulator is
              if (i >= p.slots && !wait(&s_done[slot], ph ^ 1u, s_wait, kSiteEmpty)) {
                alive = false;
                break;
              }
              const uint32_t ws = sw + slot * p.stage_bytes;
              mbar_arrive_expect_tx(&s_full[slot], p.stage_bytes);
              if constexpr (kTrans) {
                tma_load3(ws, &p.wmap, &s_full[slot], u * 64, 0, g);
              } else {
                for (int c = 0; c < kt; ++c)
                  tma_load3(ws + c * 8192, &p.wmap, &s_full[slot], c * 64, u * 64, g);
              }
              if (++slot == p.slots) {
                slot = 0;
                ph ^= 1u;
              }
            }
          }
          *s_w = i;
        }
      }
      cp_wait_all();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (s_wait->gave_up && tid == 0) {  // warp 9 issues base's and H's copies, its and warp 10's arrivals count
      land_ring(s_full, p.slots, *s_w, [](int) { return 0; });
      land_ring(s_bfull, p.bslots, s_units[0], [&](int step) { return s_units[1] <= step ? 32 : 0; });
      land_ring(s_hfull, p.hslots, s_items[0], [&](int step) { return s_items[1] <= step ? 32 : 0; });
    }
    __syncwarp();
    if (warp == 8) tmem_dealloc(tmem, 64 * kExpandSlots);
  }

  // Rows without adapter: base itself.
  pdl_wait();
  if (p.base == p.y) return;
  const int bare = p.offsets[p.count];
  const int64_t pieces = static_cast<int64_t>(p.b - bare) * (p.n / 8);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kExpandThreads + tid; i < pieces;
       i += static_cast<int64_t>(gridDim.x) * kExpandThreads) {
    const int64_t rr = i / (p.n / 8);
    const int64_t at = static_cast<int64_t>(p.order[bare + rr]) * p.n + (i - rr * (p.n / 8)) * 8;
    st_stream(p.y + at, p.base ? ld_stream(p.base + at) : make_uint4(0, 0, 0, 0));
  }
}

// ------------------------------------------------------------------- outer
struct OuterArgs {
  CUtensorMap map;   // Z: 128 rows x 64 columns
  CUtensorMap hmap;  // H: 128 rows x 64 of r
  CUtensorMap wmap;  // kDual: W: 128 rows of k x 64 of r
  const int4* tiles;
  const int32_t* order;
  const int32_t* first128;  // tiles of 128 rows before each group; [count]: all with adapter
  int cap16, count;
  const uint16_t* z;
  int64_t ldz;
  const int8_t* q;
  const float* sq;
  const uint16_t* h;  // b x r, or (kByRank) b x 2 r, two terms (store_value)
  const float* scale; // or null: 1
  uint16_t* out;      // count x k x r, or (kByRank) count x r x k
  float* part;        // 2 gridDim.y slots shaped like one group's output
  float* dpart;       // kDual: gridDim.x x b x r sums
  int64_t b;
  int k, r;
  int hr, rp;         // columns of H: r or 2 r; rounded up to 16
  int stages, htiles; // Z stages, H tiles in shared memory
  int dcol;           // kDual: first tensor-memory column of the two row accumulators
  uint32_t tmem_cols;
  bool zeros;         // one chunk: no sum kernel follows, which would write them
  uint64_t wait_ns;
  int stall;          // self-test: one of the warps that load Z stops at once
};

// Warps: 8 that load Z (16 convert codes: 8 of them took 0.9 us for a block that HBM delivers in
// 0.4), then MMA, 4 that drain, 2 that load H and W, MMA of dh.
__host__ __device__ constexpr int outer_z_warps(bool codes) { return codes ? 16 : 8; }
__host__ __device__ constexpr int outer_threads(bool codes) { return 32 * (outer_z_warps(codes) + 8); }
constexpr int kOuterStages = 4;     // at most
// Steps of 128 x 128 codes under way to a block, in registers' stead. 2 us pass between a request
// and its data while HBM is busy: 3 steps of 16 KB are 24 of the 44 KB per us that an SM can get.
constexpr int kOuterAhead = 5;
constexpr int kOuterRawStep = 16384 + 512;  // codes; a scale for each row

// A slice of Z's 128-column blocks (blockIdx.x), the row tiles of chunk blockIdx.y. Tiles of one
// group form a run, summed in tensor memory (lane = column of Z, column = rank). A run that
// is its whole group is rounded into `out`; one that the chunk's ends cut leaves its fp32
// sums in the chunk's slot (0: the run starts the chunk, else 1) for the sum kernel, in the
// order [block][rank / 4][column of the block][4], in which a warp writes 512 bytes at a time
// (rows of the output would be 32 pieces in 32 lines: 6 us a run at 768 columns of rank 64).
// kByRank (dA): H is dh in two BF16 terms side by side, 2 r accumulator columns, added at the end:
// rounded once to BF16, dh would put as large an error into dA as dA's own rounding, for 8 MMAs
// of a few more columns.
// kDual (r <= 64): the same Z stage also serves the product over its columns, dh = Z W: a
// tile's 128 x r sums over this slice go to `dpart` ([slice][rank / 4][position][4]), and dY is
// read once for both gradients. One block on an SM, for the accumulators and for as few slices, so
// parts of dh, as they allow. 8192 x 25600, rank 64: 92 us, 420 MB of dY read and 71 MB of parts of
// dh written, of which 52 reach DRAM before they are added up (5.1 TB/s); X, 8192 x 5120: 26 us; X
// in codes, 8192 x 4096, rank 32: 28 us, where each step's loads, conversion and products wait for
// one another (the conversion alone would take the integer pipe 3.3 us).
template <bool kCodes, bool kByRank, bool kDual>
__global__ void __launch_bounds__(outer_threads(kCodes), 1) outer_kernel(const __grid_constant__ OuterArgs p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_full[kOuterStages], s_empty[kOuterStages], s_hfull[kOuterStages],
      s_hempty[kOuterStages], s_dfull[2], s_dfree[2], s_run, s_free, s_end;
  __shared__ uint32_t s_tmem;
  __shared__ WaitState s_wait;
  __shared__ int s_z[kCodes ? 1 : 8], s_w, s_h[2];  // steps of each warp that loads Z; of W; tiles of H
  constexpr int kStage = 32768 + (kDual ? 16384 : 0);
  constexpr int kZ = outer_z_warps(kCodes), kMma = kZ, kDrain = kZ + 1, kLoad = kZ + 5, kMma2 = kZ + 7;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  const int total = p.first128[p.count];
  const int chunks = min(static_cast<int>(gridDim.y), total);  // none of them empty
  if (total == 0) {  // no rows with an adapter at all
    pdl_wait();
    if (blockIdx.x == 0 && p.zeros)
      for (int64_t i = tid; i < static_cast<int64_t>(p.count) * p.k * p.r / 8; i += blockDim.x)
        reinterpret_cast<uint4*>(p.out)[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  if (static_cast<int>(blockIdx.y) >= chunks) {
    pdl_wait();
    return;
  }
  const int begin = chunk_begin(blockIdx.y, chunks, total);
  const int end = chunk_begin(blockIdx.y + 1, chunks, total);
  const int blk0 = blockIdx.x * (p.k / 128) / gridDim.x;
  const int nb = (blockIdx.x + 1) * (p.k / 128) / gridDim.x - blk0;
  const int stages = p.stages;
  uint8_t* smem = align1k(smem_raw);
  const uint32_t sz = smem_u32(smem);
  const int hbytes = (p.rp + 63) / 64 * 16384;
  const uint32_t sh = sz + stages * kStage;        // p.htiles H tiles
  const uint32_t sraw = sh + p.htiles * hbytes;    // kCodes: kOuterAhead steps
  const int4* tiles = p.tiles + 1 + p.cap16;
  if (tid == 0) {
    for (int i = 0; i < kOuterStages; ++i) {
      mbar_init(&s_full[i], (kCodes ? kZ : 256) + (kDual ? 1 : 0));
      mbar_init(&s_empty[i], kDual ? 2 : 1);
      mbar_init(&s_hfull[i], 64);
      mbar_init(&s_hempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_dfull[i], 1);
      mbar_init(&s_dfree[i], 4);
    }
    mbar_init(&s_end, kDual ? 2 : 1);
    mbar_init(&s_run, 1);
    mbar_init(&s_free, 4);
    s_wait.gave_up = 0;
    s_wait.ns = p.wait_ns;
    fence_barrier_init();
  }
  if (warp == kMma) {
    tmem_alloc(&s_tmem, p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int steps = (end - begin) * nb;
  // The grouping and Z are read before the kernel in front has ended: no kernel of the same call
  // writes them.
  if (warp < kZ) {
    constexpr int kRows = 128 / (kZ * 4);   // rows r0 + kZ * 4 j, chunk ch (or 16 codes)
    // Eight lanes: a row, or, with codes, two rows of four chunks, which go to even chunks of one and
    // odd ones of the other (of one row the eight would meet in four).
    const int r0 = kCodes ? warp * 4 + (lane >> 4) * 2 + (lane >> 2 & 1) : tid >> 3;
    const int ch = kCodes ? (lane >> 3 & 1) * 4 + (lane & 3) : tid & 7;
    RowsAhead<kRows> ra;  // position of the loads: its tile, and the block in it
    ra.start(tiles, p.order, Items{begin, 1, 1, end - begin}, r0, kZ * 4);
    int lblk = 0;
    auto advance = [&]() {
      if (++lblk == nb) {
        lblk = 0;
        ra.advance();
      }
    };
    int rs = 0;  // raw slot of the next fetch, the one that the current step has just read
    auto fetch = [&]() {
      if (ra.at < end - begin) {
        const uint32_t at = sraw + rs * kOuterRawStep + tid * 16;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          const int64_t row = max(ra.row[j], 0);
          cp16(at + j * (kZ * 512), p.q + row * p.k + (blk0 + lblk) * 128 + ch * 16, ra.row[j] >= 0);
        }
        // the warp's rows, one lane each
        int srow = -1;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          const int other = __shfl_sync(0xFFFFFFFFu, ra.row[j], (lane & 2) * 8 + (lane & 1) * 4);
          if (lane >> 2 == j) srow = other;
        }
        if (lane < 4 * kRows)
          cp4(sraw + rs * kOuterRawStep + 16384 + (warp * 4 + (lane & 3) + (lane >> 2) * kZ * 4) * 4,
              p.sq + static_cast<int64_t>(max(srow, 0)) * (p.k >> 7) + blk0 + lblk, srow >= 0);
        advance();
      }
      cp_commit();
      if (++rs == kOuterAhead) rs = 0;
    };
    if constexpr (kCodes) {
      for (int a = 0; a < kOuterAhead; ++a) fetch();
    }
    int slot = 0, step = 0;
    uint32_t phase = 0;
    for (; step < steps; ++step) {
      if (p.stall && warp == 1) break;
      uint4 v[kRows];
      float sc[kRows];
      if constexpr (kCodes) {
        cp_wait<kOuterAhead - 1>();
        __syncwarp();  // the scales came by other lanes of the warp
        const uint32_t at = sraw + rs * kOuterRawStep + tid * 16;
        const uint32_t st = sraw + rs * kOuterRawStep + 16384 + r0 * 4;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          v[j] = lds16(at + j * (kZ * 512));
          sc[j] = lds4(st + j * (kZ * 16));
        }
        __syncwarp();  // before a lane's next copies take their place
      }
      if (step >= stages && !warp_wait(&s_empty[slot], phase ^ 1u, &s_wait, kSiteEmpty)) break;
      const uint32_t zs = sz + slot * kStage;
      if constexpr (kCodes) {
        const uint32_t half = zs + (ch >> 2) * 16384;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          uint4 lo, hi;
          dequant16(v[j], sc[j], lo, hi);
          sts16(half + sw128(r0 + kZ * 4 * j, 2 * (ch & 3)), lo);
          sts16(half + sw128(r0 + kZ * 4 * j, 2 * (ch & 3) + 1), hi);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_full[slot]);
        fetch();
      } else {
        if (ra.run >= 0 && ra.count == 128) {
          if (tid == 0) {
            mbar_arrive_expect_tx(&s_full[slot], 32768);
            const uint64_t once = read_once_policy();
            tma_load_once(zs, &p.map, &s_full[slot], (blk0 + lblk) * 128, ra.run, once);
            tma_load_once(zs + 16384, &p.map, &s_full[slot], (blk0 + lblk) * 128 + 64, ra.run, once);
          }
          if (lane == 0) mbar_arrive_n(&s_full[slot], tid == 0 ? 31 : 32);
        } else {
#pragma unroll
          for (int j = 0; j < kRows; ++j)
#pragma unroll
            for (int half = 0; half < 2; ++half)
              if (r0 + kZ * 4 * j < (ra.count + 15) / 16 * 16)
                cp16(zs + half * 16384 + sw128(r0 + kZ * 4 * j, ch),
                     p.z + max(ra.row[j], 0) * p.ldz + (blk0 + lblk) * 128 + half * 64 + ch * 8,
                     ra.row[j] >= 0);
          cp_arrive(&s_full[slot]);
        }
        advance();
      }
      if (++slot == stages) {
        slot = 0;
        phase ^= 1u;
      }
    }
    if (!kCodes && lane == 0) s_z[kCodes ? 0 : warp] = step;
    cp_wait_all();
  } else if (warp == kMma) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(p.rp) | kAMajorMn | kBMajorMn;
      int runs = 0, slot = 0, hs = 0;
      uint32_t phase = 0, hphase = 0;
      bool alive = true;
      bool fresh = true;
      int run_end = min(end, p.first128[tiles[begin].x + 1]);
      int rows = tiles[begin].z;
      for (int tile = begin; tile < end && alive; ++tile) {
        const uint32_t hb = desc_mn(sh + hs * hbytes, 16384);
        const int ksteps = (rows + 15) / 16;
        if (tile + 1 < end) rows = tiles[tile + 1].z;
        alive = wait(&s_hfull[hs], hphase, &s_wait, kSiteFull);
        if (!alive) break;
        for (int b = 0; b < nb; ++b) {
          if (!wait(&s_full[slot], phase, &s_wait, kSiteFull)) {
            alive = false;
            break;
          }
          fence_proxy_async_smem();
          tc_fence_after();
          const uint32_t za = desc_mn(sz + slot * kStage, 16384), d = tmem + b * p.rp;
          mma(d, za, hb, idesc, !fresh);
#pragma unroll
          for (int k = 1; k < 8; ++k)  // 16 rows each, as far as the tile has any
            if (k < ksteps) mma(d, za + k * 128, hb + k * 128, idesc, true);
          mma_commit(&s_empty[slot]);
          if (++slot == stages) {
            slot = 0;
            phase ^= 1u;
          }
        }
        if (!alive) break;
        mma_commit(&s_hempty[hs]);
        if (++hs == p.htiles) {
          hs = 0;
          hphase ^= 1u;
        }
        fresh = tile + 1 == run_end;
        if (fresh) {
          mma_commit(&s_run);
          if (run_end < end) {
            run_end = min(end, p.first128[tiles[run_end].x + 1]);
            alive = wait(&s_free, runs & 1, &s_wait, kSiteAccEmpty);
          }
          ++runs;
          tc_fence_after();
        }
      }
      mma_commit(&s_end);
      wait_mmas(&s_end);
    }
  } else if (warp == kMma2) {
    // An MMA of so few columns takes its issuer 60 to 100 cycles whatever its size, so the row
    // sums have an issuer of their own.
    if (kDual && lane == 0) {
      const uint32_t didesc = idesc_bf16(p.rp) | kBMajorMn;
      int slot = 0;
      uint32_t phase = 0;
      bool alive = true;
      for (int nth = 0; nth < end - begin && alive; ++nth) {
        const uint32_t dacc = tmem + p.dcol + (nth & 1) * p.rp;
        if (nth >= 2 && !wait(&s_dfree[nth & 1], ((nth >> 1) & 1) ^ 1u, &s_wait, kSiteAccEmpty)) break;
        for (int b = 0; b < nb; ++b) {
          if (!wait(&s_full[slot], phase, &s_wait, kSiteFull)) {
            alive = false;
            break;
          }
          fence_proxy_async_smem();
          tc_fence_after();
          const uint32_t za = desc_k(sz + slot * kStage), wa = desc_mn(sz + slot * kStage + 32768, 0);
          mma(dacc, za, wa, didesc, b > 0);
#pragma unroll
          for (int k = 1; k < 8; ++k)  // 16 columns each
            mma(dacc, za + (k >> 2) * 1024 + (k & 3) * 2, wa + k * 128, didesc, true);
          mma_commit(&s_empty[slot]);
          if (++slot == stages) {
            slot = 0;
            phase ^= 1u;
          }
        }
        if (alive) mma_commit(&s_dfull[nth & 1]);
      }
      mma_commit(&s_end);
      wait_mmas(&s_end);
    }
  } else if (warp >= kDrain && warp < kLoad) {
    const int sub = warp & 3;  // tensor-memory lanes of this warp
    const uint32_t lanes = static_cast<uint32_t>(sub * 32) << 16;
    const int64_t size = static_cast<int64_t>(p.k) * p.r;
    pdl_wait();  // the kernels before may still read or write what this one writes
    if (p.zeros && blockIdx.y == 0)
      for (int g = 0; g < p.count; ++g) {  // adapters without rows
        if (p.first128[g] != p.first128[g + 1]) continue;
        uint4* out = reinterpret_cast<uint4*>(p.out + g * size);
        const int l = tid - kDrain * 32, per = kByRank ? nb * 16 : nb * 16 * p.r;
        for (int i = l; i < (kByRank ? per * p.r : per); i += 128)
          out[kByRank ? static_cast<int64_t>(i / per) * (p.k / 8) + blk0 * 16 + i % per
                      : static_cast<int64_t>(blk0) * 16 * p.r + i] = make_uint4(0, 0, 0, 0);
      }
    int runs = 0;
    bool alive = true;
    for (int tile = begin; tile < end && alive;) {
      const int g = tiles[tile].x;
      const int first = tile;
      const int gb = p.first128[g], ge = p.first128[g + 1];
      const int stop = min(end, ge);
      const float f = p.scale ? p.scale[g] : 1.0f;
      if constexpr (kDual) {
        for (; tile < stop; ++tile) {
          const int nth = tile - begin;
          const int4 t = tiles[tile];
          if (!warp_wait(&s_dfull[nth & 1], (nth >> 1) & 1, &s_wait, kSiteDrain)) {
            alive = false;
            break;
          }
          tc_fence_after();
          const int i = sub * 32 + lane;
          float* dst = p.dpart + (static_cast<int64_t>(blockIdx.x) * p.r * p.b + (t.y + i) * 4);
          for (int c = 0; c < p.rp; c += 16) {
            uint32_t v[16];
            tmem_ld16(tmem + lanes + p.dcol + (nth & 1) * p.rp + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int u = 0; u < 16; u += 4)
              if (i < t.z && c + u < p.r)
                *reinterpret_cast<float4*>(dst + (c + u) * p.b) =
                    make_float4(f * __uint_as_float(v[u]), f * __uint_as_float(v[u + 1]),
                                f * __uint_as_float(v[u + 2]), f * __uint_as_float(v[u + 3]));
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_dfree[nth & 1]);
        }
        if (!alive) break;
      }
      tile = stop;
      if (!warp_wait(&s_run, runs & 1, &s_wait, kSiteDrain)) break;
      ++runs;
      tc_fence_after();
      const bool whole = first == gb && stop == ge;
      float* part = p.part + (2 * blockIdx.y + (first == begin ? 0 : 1)) * size;
      uint16_t* out = p.out + g * size;
      for (int b = 0; b < nb; ++b) {
        const int64_t j = (blk0 + b) * 128 + sub * 32 + lane;
        float* quads = part + static_cast<int64_t>(blk0 + b) * 128 * p.r + (sub * 32 + lane) * 4;
        for (int c = 0; c < p.r; c += 8) {
          uint32_t v[8], w[8];
          tmem_ld8(tmem + lanes + b * p.rp + c, v);
          if (kByRank) tmem_ld8(tmem + lanes + b * p.rp + p.r + c, w);
          tmem_wait_ld();
          float o[8];
#pragma unroll
          for (int u = 0; u < 8; ++u)
            o[u] = f * (kByRank ? both_terms(__uint_as_float(v[u]), __uint_as_float(w[u])) : __uint_as_float(v[u]));
          if (!whole) {
            *reinterpret_cast<float4*>(quads + c * 128) = make_float4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<float4*>(quads + (c + 4) * 128) = make_float4(o[4], o[5], o[6], o[7]);
          } else if (kByRank) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              out[(c + e) * static_cast<int64_t>(p.k) + j] = static_cast<uint16_t>(pack2(o[e], 0.0f));
          } else {
            *reinterpret_cast<uint4*>(out + j * p.r + c) = make_uint4(
                pack2(o[0], o[1]), pack2(o[2], o[3]), pack2(o[4], o[5]), pack2(o[6], o[7]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_free);
    }
  } else {
    const int l = tid - kLoad * 32, rchunks = p.rp / 8;
    const int hr = l >> 3, hc = l & 7;  // H: rows hr + 8 j, chunks hc, hc + 8
    int slot = 0, hs = 0, step = 0, loaded = 0;
    uint32_t phase = 0, hphase = 0;
    bool alive = true;
    RowsAhead<16> ra;
    ra.start(tiles, p.order, Items{begin, 1, 1, end - begin}, hr, 8);
    pdl_wait();
    for (int tile = begin; tile < end && alive; ++tile) {
      if (tile - begin >= p.htiles && !warp_wait(&s_hempty[hs], hphase ^ 1u, &s_wait, kSiteHEmpty))
        break;
      if (ra.run >= 0 && ra.count == 128) {
        if (l == 0) {
          mbar_arrive_expect_tx(&s_hfull[hs], hbytes);
          for (int c = 0; c < hbytes / 16384; ++c)
            tma_load(sh + hs * hbytes + c * 16384, &p.hmap, &s_hfull[hs], c * 64, ra.run);
        }
        if (lane == 0) mbar_arrive_n(&s_hfull[hs], l == 0 ? 31 : 32);
      } else {
        for (int c = hc; c < rchunks; c += 8)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (hr + 8 * j >= (ra.count + 15) / 16 * 16) break;
            const bool in = ra.row[j] >= 0 && c * 8 < p.hr;
            cp16(sh + hs * hbytes + (c >> 3) * 16384 + sw128(hr + 8 * j, hc),
                 p.h + (in ? static_cast<int64_t>(ra.row[j]) * p.hr + c * 8 : 0), in);
          }
        cp_arrive(&s_hfull[hs]);
      }
      if (++hs == p.htiles) {
        hs = 0;
        hphase ^= 1u;
      }
      ++loaded;
      const int group = ra.group;
      ra.advance();
      if (kDual && warp == kLoad) {  // one warp alone, as the copies of W are its own
        for (int b = 0; b < nb; ++b, ++step) {
          if (step >= stages && !warp_wait(&s_empty[slot], phase ^ 1u, &s_wait, kSiteEmpty)) {
            alive = false;
            break;
          }
          if (l == 0) {
            mbar_arrive_expect_tx(&s_full[slot], 16384);
            tma_load3(sz + slot * kStage + 32768, &p.wmap, &s_full[slot], 0, (blk0 + b) * 128, group);
          }
          if (++slot == stages) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
    }
    if (lane == 0) {
      s_h[warp - kLoad] = loaded;
      if (warp == kLoad) s_w = step;
    }
    cp_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (s_wait.gave_up && tid == 0) {
    if constexpr (!kCodes)  // Z comes by warp 0's TMA, W by kLoad's; whichever went further
      land_ring(s_full, stages, max(s_z[0], s_w), [&](int at) {
        int missing = kDual && s_w <= at ? 1 : 0;
        for (int w = 0; w < kZ; ++w) missing += s_z[w] <= at ? 32 : 0;
        return missing;
      });
    land_ring(s_hfull, p.htiles, s_h[0], [&](int at) { return s_h[1] <= at ? 32 : 0; });
  }
  __syncwarp();
  if (warp == kMma) tmem_dealloc(tmem, p.tmem_cols);
}

// -------------------------------------------------------------------- host
int tiles_estimate(const AdapterCall& c) {
  // full tiles and half a partial one per adapter
  return std::max(1, std::min(row_tiles_cap(c.g.b, c.g.count, 128), c.g.b / 128 + (c.g.count + 1) / 2));
}

template <typename Args>
cudaError_t launch(void (*kernel)(Args), dim3 grid, int threads, int smem, int cluster, bool pdl,
                   const Args& args, cudaStream_t st) {
  if (smem > 0) {
    const cudaError_t e = allow_smem(kernel, kMaxSmem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  int n = 0;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = cluster;
    at[n].val.clusterDim.y = 1;
    at[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A tensor map of BF16, 128-byte swizzle, boxes of 64 of the contiguous dimension.
// strides: of dimensions 1 .., in elements.
template <int kRank>
cudaError_t encode(CUtensorMap* map, const uint16_t* base, const int64_t (&dims)[kRank],
                   const int64_t (&strides)[kRank - 1], const int (&box)[kRank]) {
  static std::atomic<EncodeTiledFn> known{nullptr};
  EncodeTiledFn fn = known.load(std::memory_order_acquire);
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
    fn = reinterpret_cast<EncodeTiledFn>(f);
    known.store(fn, std::memory_order_release);
  }
  cuuint64_t d[kRank], s[kRank];
  cuuint32_t b[kRank], one[kRank];
  for (int i = 0; i < kRank; ++i) {
    d[i] = static_cast<cuuint64_t>(dims[i]);
    b[i] = static_cast<cuuint32_t>(box[i]);
    one[i] = 1;
    if (i > 0) s[i - 1] = static_cast<cuuint64_t>(strides[i - 1]) * 2;
  }
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kRank, const_cast<uint16_t*>(base), d, s, b, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}
// rows x cols, row stride ld, boxes of `high` rows.
cudaError_t encode_rows(CUtensorMap* map, const uint16_t* base, int64_t rows, int64_t cols, int64_t ld,
                        int high = 128) {
  return encode<2>(map, base, {cols, rows}, {ld}, {64, high});
}

// Up to three turns of its blocks, the expand kernel adds up what the last outer product left, while
// its first copies are under way: a launch less (gradients of 4096 x 4096, rank 16: 53 instead of
// 55.5 us; 8192 x 5120, rank 64, 640 blocks: 184 instead of 185). More are a launch of their own,
// with eight blocks on an SM instead of two.
constexpr int kMaxExpandSums = 3 * 2 * kSms;

int round16(int r) { return (r + 15) / 16 * 16; }

// Never launched: a kernel of the shrink kernels' shape that allocates no tensor memory. For one
// that does, the occupancy calls answer one block per SM; two of at most 256 columns do run there.
__global__ void __launch_bounds__(kShrinkThreads, 2) shrink_shape_kernel(int* out) {
  extern __shared__ int shape_smem[];
  if (out) out[0] = shape_smem[threadIdx.x];
}
// The cluster size for `tiles` row tiles of a shrink kernel with `smem` bytes of shared memory
// (kind, rank16: what smem depends on): at most 8 blocks, as many as let all clusters run at once (a
// cluster keeps within a GPC: 33 clusters of 7 fit, or 44 of 6, and a second wave doubles the time:
// 45 against 25 us for 38 tiles of codes); one cluster in 20 may come late.
// How many fit is asked once per device, under a lock, and only an answer is kept: the size sets the
// order of the sums, so it must not depend on which call comes first or on which thread.
cudaError_t cluster_size(int tiles, int kind, int rank16, int smem, int* size) {
  constexpr int kDevices = 64;
  static std::mutex mu;
  static int known[kDevices][3][9][9];  // clusters that fit, plus 1; 0: not asked yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  for (*size = 8; *size > 1; --*size) {
    int fit = dev < kDevices ? known[dev][kind][*size][rank16] - 1 : -1;
    if (fit < 0) {
      e = allow_smem(shrink_shape_kernel, kMaxSmem);
      if (e != cudaSuccess) return e;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(*size, 2 * kSms);
      cfg.blockDim = dim3(kShrinkThreads);
      cfg.dynamicSmemBytes = smem + 1024;  // and the kernels' static part
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = *size;
      at[0].val.clusterDim.y = 1;
      at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&fit, shrink_shape_kernel, &cfg);
      if (e != cudaSuccess) {
        cudaGetLastError();  // returned here; not a later launch's error
        return e;
      }
      if (dev < kDevices) known[dev][kind][*size][rank16] = fit + 1;
    }
    if (int64_t(tiles) * 20 <= int64_t(fit) * 21) break;
  }
  return cudaSuccess;
}

// trans: W is count x k x r (the backward pass's B).
cudaError_t launch_shrink(const AdapterCall& c, bool trans, const uint16_t* z, int64_t ldz, int k,
                          const uint16_t* w, const float* scale, uint16_t* out, cudaStream_t st) {
  const bool codes = !trans && c.xq8;
  const int rp = round16(c.r);
  ShrinkArgs p{{}, {}, {}, c.g.tiles, c.g.order, small_tiles_cap(c.g.b, c.g.count), z, ldz,
               codes ? c.xq8 : nullptr, codes ? c.sx : nullptr, scale, out, k, c.r, rp, trans, 0, 0};
  // Two blocks per SM: 110 KB each, of which the parts need 128 x (rp + 4) fp32. As many W as Z
  // stages; with codes two raw groups a team (one beyond rank 64) and the rest for W, whose copies
  // take 2 us and more while HBM is busy.
  const int wbytes = trans ? (rp + 63) / 64 * 8192 : rp * 128, per = codes ? 2 : 1;
  p.stages = codes ? (rp > 64 ? 1 : 2)
                   : std::max(2, std::min(kShrinkStages, 110 * 1024 / (16384 + wbytes)));
  p.wstages = codes ? std::min(kShrinkStages, (110 * 1024 - p.stages * 32768) / (2 * wbytes)) : p.stages;
  const int smem = std::max(per * (p.stages * 16384 + p.wstages * wbytes), 128 * (rp + 4) * 4) + 1024;
  p.wait_ns = c.wait_ns;
  p.stall = c.stall;
  auto kernel = trans ? shrink_kernel<false, true>
                      : (codes ? shrink_kernel<true, false> : shrink_kernel<false, false>);
  int splits = 1;  // blocks of a cluster, over which the reduction is split
  cudaError_t e = cluster_size(tiles_estimate(c), trans ? 2 : codes, rp / 16, smem, &splits);
  if (e != cudaSuccess) return e;
  const dim3 grid(splits, row_tiles_cap(c.g.b, c.g.count, 128));
  e = trans ? encode<3>(&p.wmap, w, {c.r, k, c.g.count}, {c.r, int64_t(c.r) * k}, {64, 64, 1})
            : encode_rows(&p.wmap, w, int64_t(c.g.count) * c.r, k, k, rp);
  if (e == cudaSuccess && !codes) e = encode_rows(&p.map, z, c.g.b, k, ldz);
  if (e == cudaSuccess && !codes) e = encode_rows(&p.map16, z, c.g.b, k, ldz, 16);
  // a pair of codes as one element: the copies are the same bytes
  if (e == cudaSuccess && codes)
    e = encode_rows(&p.map, reinterpret_cast<const uint16_t*>(c.xq8), c.g.b, k / 2, k / 2, 32);
  if (e != cudaSuccess) return e;
  return launch(kernel, grid, kShrinkThreads, smem, splits, false, p, st);
}

int sum_blocks(const SumArgs& p) { return p.dh_blocks + (p.side[0].blocks + p.side[1].blocks) * p.count; }

cudaError_t launch_expand(const AdapterCall& c, bool trans, const uint16_t* h, int ldh, const uint16_t* w,
                          int n, const float* scale, uint16_t* y, const SumArgs& sum, bool pdl,
                          cudaStream_t st) {
  const int rp = round16(c.r), kt = (rp + 63) / 64;
  ExpandArgs p{{}, {}, {}, {}, c.g.tiles, c.g.order, small_tiles_cap(c.g.b, c.g.count), h, scale, c.base, y,
               first128_of(c.g), c.g.offsets, c.g.b, c.g.count, n, c.r, rp, ldh, 0, 0, 0, 0, 1, sum, sum_blocks(sum)};
  // Two blocks per SM, 112 KB each: 4 stages of W and of base and a second H tile as far as they
  // fit (W's copies take 2 us and more while HBM is busy), 2 of each beyond rank 64.
  p.stage_bytes = trans ? rp * 128 : kt * 8192;
  p.slots = kt == 1 ? kExpandSlots : 2;
  p.bslots = kt == 1 ? kBaseSlots : 2;
  const int rest = p.slots * p.stage_bytes + p.bslots * 16384;
  p.hslots = rest + 2 * kt * 16384 <= 112 * 1024 ? 2 : 1;
  const int fixed = p.hslots * kt * 16384 + p.slots * p.stage_bytes;
  const int smem = fixed + p.bslots * 16384 + kExpandBars;
  p.wait_ns = c.wait_ns;
  p.stall = c.stall;
  const int64_t r = c.r;
  cudaError_t e =
      trans ? encode<3>(&p.wmap, w, {n, r, c.g.count}, {n, r * n}, {64, rp, 1})
            : encode<3>(&p.wmap, w, {r, n, c.g.count}, {r, r * n}, {64, 64, 1});
  if (e == cudaSuccess) e = encode_rows(&p.hmap, h, c.g.b, r, ldh);
  if (e == cudaSuccess && c.base) e = encode_rows(&p.map, c.base, c.g.b, n, n);
  if (e == cudaSuccess && c.base) e = encode_rows(&p.map16, c.base, c.g.b, n, n, 16);
  if (e != cudaSuccess) return e;
  // Parts of a row tile: 4 to 12 units, so that the last turn of the blocks is nearly full (an
  // item costs about one unit more than it has, for its H).
  const int units = n / 64, tiles = tiles_estimate(c);
  int64_t cost = INT64_MAX;
  for (int s = std::max(1, units / 12); s <= std::max(1, units / 4); ++s) {
    const int64_t turns = (int64_t(tiles) * s + 2 * kSms - 1) / (2 * kSms);
    const int64_t all = turns * (1 + (units + s - 1) / s);
    if (all < cost) cost = all, p.segs = s;
  }
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(
      2 * kSms, std::max<int64_t>(p.sums, int64_t(row_tiles_cap(c.g.b, c.g.count, 128)) * p.segs)));
  auto kernel = p.sums ? expand_kernel<true, true>
                       : (trans ? expand_kernel<true, false> : expand_kernel<false, false>);
  return launch(kernel, dim3(blocks), kExpandThreads, smem, 1, pdl, p, st);
}

// Column blocks and row chunks of the outer kernel: one thread block per SM, the split that
// moves the fewest bytes through the busiest block (Z, H again for every slice, parts).
struct OuterPlan {
  int slices, chunks, stages, htiles, dcol;
  uint32_t cols;
};
// What a block could have moved in the time of one more launch (the sum kernel's).
constexpr double kLaunchBytes = 110e3;

// hr: columns of H.
OuterPlan outer_plan(int64_t b, int64_t count, int k, int hr, bool codes, bool dual) {
  const int rp = round16(hr), blocks = k / 128;
  const int tiles = static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>(row_tiles_cap(b, count, 128), b / 128 + (count + 1) / 2)));
  OuterPlan best{};
  double cost = 1e30;
  for (int nb = 1; nb <= 512 / rp - (dual ? 2 : 0) && nb <= blocks; ++nb) {
    const int slices = (blocks + nb - 1) / nb;
    for (int chunks : {std::max(1, std::min(tiles, kSms / slices)), 1}) {
    const double waves = double((int64_t(slices) * chunks + kSms - 1) / kSms);
    const double each = double((tiles + chunks - 1) / chunks) *
                            (nb * 32768.0 + 256.0 * rp + (dual ? 512.0 * rp : 0.0)) +
                        (chunks > 1 ? 2.0 * nb * 128 * rp * 4 + kLaunchBytes : 0.0);
    const double all = waves * each + (dual ? double(slices) * tiles * 512 * rp / kSms : 0.0);
    if (all < cost) {
      cost = all;
      best.slices = slices;
      best.chunks = chunks;
      best.dcol = nb * rp;
    }
    }
  }
  const int used = best.dcol + (dual ? 2 * rp : 0);
  best.cols = 32;
  while (static_cast<int>(best.cols) < used) best.cols *= 2;
  // As many H tiles as the Z stages reach ahead (nb_min: the blocks of the smallest slice).
  const int nb_min = blocks / best.slices, hbytes = (rp + 63) / 64 * 16384;
  const int stage = 32768 + (dual ? 16384 : 0), raw = codes ? kOuterAhead * kOuterRawStep : 0;
  for (best.stages = codes ? 2 : kOuterStages; best.stages > 1; --best.stages) {
    best.htiles = std::max(2, 1 + (best.stages - 1 + nb_min - 1) / nb_min);
    if (best.stages * stage + best.htiles * hbytes + raw <= 224 * 1024) return best;
  }
  best.stages = 2;  // codes beyond rank 64: one H tile of 64 KB
  best.htiles = 1;
  return best;
}

template <bool kCodes, bool kByRank, bool kDual>
cudaError_t launch_outer(const AdapterCall& c, const OuterPlan& plan, const uint16_t* z, int64_t ldz,
                         int k, const uint16_t* h, const float* scale, uint16_t* out, float* part,
                         float* dpart, bool pdl, cudaStream_t st) {
  const int hr = kByRank ? 2 * c.r : c.r, rp = round16(hr);
  const int cap16 = small_tiles_cap(c.g.b, c.g.count);
  OuterArgs p{{}, {}, {}, c.g.tiles, c.g.order, first128_of(c.g), cap16, c.g.count, z, ldz, c.xq8, c.sx, h, scale,
              out, part, dpart, c.g.b, k, c.r, hr, rp, plan.stages, plan.htiles, plan.dcol, plan.cols, plan.chunks == 1,
              c.wait_ns, c.stall};
  cudaError_t e = encode_rows(&p.hmap, h, c.g.b, hr, hr);
  if (e == cudaSuccess && !kCodes) e = encode_rows(&p.map, z, c.g.b, k, ldz);
  if (e == cudaSuccess && kDual)
    e = encode<3>(&p.wmap, c.bm, {c.r, k, c.g.count}, {c.r, int64_t(c.r) * k}, {64, 128, 1});
  if (e != cudaSuccess) return e;
  const int smem = plan.stages * (32768 + (kDual ? 16384 : 0)) +
                   plan.htiles * ((rp + 63) / 64) * 16384 + (kCodes ? kOuterAhead * kOuterRawStep : 0) +
                   1024;
  return launch(outer_kernel<kCodes, kByRank, kDual>, dim3(plan.slices, plan.chunks), outer_threads(kCodes),
                smem, 1, pdl, p, st);
}

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

struct BackwardPlan {
  bool dual;  // dh and dB from one pass over dY: up to rank 64, where the row parts are small
  OuterPlan a, b;
  size_t dh, pa, pb, pd, bytes;  // workspace offsets
};
BackwardPlan backward_plan(int64_t b, int64_t m, int64_t n, int64_t r, int64_t count, bool codes) {
  BackwardPlan s;
  s.dual = r <= 64;
  s.a = outer_plan(b, count, int(m), int(2 * r), codes, false);
  s.b = outer_plan(b, count, int(n), int(r), false, s.dual);
  s.dh = 0;
  s.pa = up256(size_t(b) * 2 * r * 2);
  s.pb = s.pa + up256(size_t(2) * s.a.chunks * m * r * 4);
  s.pd = s.pb + up256(size_t(2) * s.b.chunks * n * r * 4);
  s.bytes = s.pd + (s.dual ? up256(size_t(s.b.slices) * b * r * 4) : 0);
  return s;
}

// By device; a kernel's pointer where its limit is set. More places than there are such kernels: the
// adapters', and 27 of the products on BF16 activations.
constexpr int kKnownDevices = 64, kKnownKernels = 96;
std::atomic<const void*> g_allowed[kKnownDevices][kKnownKernels];

}  // namespace

cudaError_t allow_smem(const void* kernel, int smem) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<const void*>* list = dev < kKnownDevices ? g_allowed[dev] : nullptr;
  for (int i = 0; list && i < kKnownKernels; ++i) {
    const void* k = list[i].load(std::memory_order_acquire);
    if (k == kernel) return cudaSuccess;
    if (!k) break;
  }
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (e != cudaSuccess) return e;
  for (int i = 0; list && i < kKnownKernels; ++i) {
    const void* none = nullptr;
    if (list[i].compare_exchange_strong(none, kernel, std::memory_order_acq_rel) || none == kernel) break;
  }
  return cudaSuccess;
}

void release_adapter_cache() {
  for (auto& list : g_allowed)
    for (auto& k : list) k.store(nullptr, std::memory_order_release);
}

cudaError_t read_and_clear_adapter_status(int* code) {
  cudaError_t e = cudaMemcpyFromSymbol(code, g_adapter_status, sizeof(int));
  if (e != cudaSuccess || *code == 0) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_adapter_status, &zero, sizeof(int));
}

cudaError_t launch_adapter_linear(const AdapterCall& c, cudaStream_t st) {
  if (small_batch(c.g.b, c.g.count, c.r)) return launch_adapter_small(c, st);
  cudaError_t e = launch_shrink(c, false, c.x, c.ldx, c.m, c.a, nullptr, c.h, st);
  if (e != cudaSuccess) return e;
  return launch_expand(c, false, c.h, c.r, c.bm, c.n, c.scale, c.y, SumArgs{}, true, st);
}

size_t adapter_backward_workspace(int64_t b, int64_t m, int64_t n, int64_t r, int64_t count) {
  // the plans differ only in what shared memory holds, not in slices and chunks
  return backward_plan(b, m, n, r, count, false).bytes;
}

cudaError_t launch_adapter_backward(const AdapterCall& c, cudaStream_t st) {
  const BackwardPlan s = backward_plan(c.g.b, c.m, c.n, c.r, c.g.count, c.xq8 != nullptr);
  uint8_t* ws = static_cast<uint8_t*>(c.workspace);
  uint16_t* dh = reinterpret_cast<uint16_t*>(ws + s.dh);
  float* pa = reinterpret_cast<float*>(ws + s.pa);
  float* pb = reinterpret_cast<float*>(ws + s.pb);
  float* pd = reinterpret_cast<float*>(ws + s.pd);
  const SumArgs none{c.g.tiles, c.g.order, c.g.offsets, first128_of(c.g), c.g.b, c.g.count, c.r,
                     pd, dh, s.b.slices, 0, {{pa, c.da, c.m, s.a.chunks, 0}, {pb, c.db, c.n, s.b.chunks, 0}}};
  auto sums = [&](bool with_dh, bool with_a, bool with_b) {
    SumArgs p = none;
    if (with_dh) p.dh_blocks = (c.g.b + 255) / 256 * (c.r / 4);
    if (with_a) p.side[0].blocks = static_cast<int>((int64_t(c.m) * c.r + 2047) / 2048);
    if (with_b) p.side[1].blocks = static_cast<int>((int64_t(c.n) * c.r + 2047) / 2048);
    return p;
  };
  auto add_up = [&](const SumArgs& p, bool pdl) {
    const int blocks = sum_blocks(p);
    return blocks ? launch(sum_kernel, dim3(blocks), 256, 0, 1, pdl, p, st) : cudaSuccess;
  };
  if (c.g.b == 0) return add_up(sums(false, true, true), false);  // zeros
  cudaError_t e;
  const bool a_cut = s.a.chunks > 1, b_cut = s.b.chunks > 1;
  if (s.dual) {
    e = launch_outer<false, false, true>(c, s.b, c.dy, c.n, c.n, c.h, c.scale, c.db, pb, pd, false, st);
    if (e == cudaSuccess) e = add_up(sums(true, false, b_cut), true);
  } else {
    e = launch_shrink(c, true, c.dy, c.n, c.n, c.bm, c.scale, dh, st);
    if (e == cudaSuccess)
      e = launch_outer<false, false, false>(c, s.b, c.dy, c.n, c.n, c.h, c.scale, c.db, pb, nullptr, true, st);
  }
  if (e == cudaSuccess)
    e = c.xq8 ? launch_outer<true, true, false>(c, s.a, nullptr, 0, c.m, dh, nullptr, c.da, pa, nullptr, true, st)
              : launch_outer<false, true, false>(c, s.a, c.x, c.ldx, c.m, dh, nullptr, c.da, pa, nullptr, true, st);
  SumArgs last = sums(false, a_cut, b_cut && !s.dual);
  if (sum_blocks(last) > kMaxExpandSums) {
    if (e == cudaSuccess) e = add_up(last, true);
    last = SumArgs{};
  }
  if (e != cudaSuccess) return e;
  return launch_expand(c, true, dh, 2 * c.r, c.a, c.m, nullptr, c.dx, last, true, st);
}

}  // namespace twq
