// Test harness: exposes what the host computes for launches on BF16 activations to the CPU tests. It
// compiles the kernel's own translation unit; only host code runs (no device, no launch).
#include <cuda_runtime.h>

// The devices are made up: as many as the test asks for, each with its own number of clusters that run
// at once, and a count of how often that is asked.
static int g_device = 0, g_asked = 0;
static cudaError_t fake_get_device(int* dev) {
  *dev = g_device;
  return cudaSuccess;
}
template <typename T>
static cudaError_t fake_max_clusters(int* n, T, const cudaLaunchConfig_t* cfg) {
  ++g_asked;
  *n = (200 + g_device) / static_cast<int>(cfg->attrs[0].val.clusterDim.x);
  return cudaSuccess;
}
#define cudaGetDevice fake_get_device
#define cudaOccupancyMaxActiveClusters fake_max_clusters
#include "twq_a16_sm100.cu"

namespace twq {
cudaError_t allow_smem(const void*, int) { return cudaSuccess; }
}  // namespace twq

#define TWQ_TEST extern "C" __attribute__((visibility("default")))

// Limits of a block's waits and of its wait for peers' parts, in ns.
TWQ_TEST uint64_t twq_test_a16_wait_limit(uint64_t ns, int stall, int rank) {
  return twq::wait_limit(ns, stall != 0, rank);
}
TWQ_TEST uint64_t twq_test_a16_parts_limit(uint64_t ns, int stall, int split, int steps) {
  return twq::parts_limit(ns, stall != 0, split, steps);
}

// Plans each product of a layer and of experts (all kernels there are) for device `dev`; out: how often the
// device was asked, and a sum over the plans that tells them apart.
template <int kWarps, int NT, int kMode, int kParts, bool kRouted>
static int64_t plan_one() {
  twq::A16Args a = {};
  a.K = 4096, a.n = 2048, a.f = 1024, a.b = kRouted ? 16 : 8 * NT, a.k = kRouted ? 4 : 1, a.count = kRouted ? 32 : 1;
  twq::Choice c;
  if (twq::choose<kWarps, NT, kMode, kParts, kRouted>(a, &c) != cudaSuccess) return -(int64_t(1) << 40);
  return c.p.cost * 8 + c.p.split_log + 64 * c.p.clusters;
}
template <int NT>
static int64_t plan_rows() {
  return plan_one<4, NT, twq::kModeH, 1, false>() + plan_one<4, NT, twq::kModeY, 1, false>() * 3 +
         plan_one<8, NT, twq::kModeY, 1, false>() * 5 + plan_one<4, NT, twq::kModeH, 1, true>() * 7 +
         plan_one<4, NT, twq::kModeAct, 1, true>() * 11 + plan_one<8, NT, twq::kModeAct, 1, true>() * 13 +
         plan_one<4, NT, twq::kModeH, 2, true>() * 17 + plan_one<4, NT, twq::kModePart, 2, true>() * 19 +
         plan_one<8, NT, twq::kModePart, 2, true>() * 23;
}
TWQ_TEST void twq_test_a16_plans(int dev, int64_t* out) {
  g_device = dev;
  g_asked = 0;
  out[1] = plan_rows<1>() + 29 * plan_rows<2>() + 31 * plan_rows<4>();
  out[0] = g_asked;
}

// One cluster's jobs and its blocks' shares, as the kernel computes them. begin: 2^log + 1 places; of each block
// (2^log places): owner, the block that gets its first job's part, or -1; others, how many blocks may send it
// parts of its last job. Returns the first job | the one behind the last << 32.
TWQ_TEST int64_t twq_test_a16_shares(int jobs, int clusters, int cluster, int per, int log, int* begin, int* owner,
                                     int* others) {
  const twq::Shares s(jobs, clusters, cluster, per, log);
  for (int r = 0; r <= 1 << log; ++r) begin[r] = s.begin(r);
  for (int r = 0; r < 1 << log; ++r) {
    const int lo = s.begin(r), hi = s.begin(r + 1);
    owner[r] = s.any(r) && lo % per ? s.owner(r, lo - lo % per) : -1;
    others[r] = 0;
    if (s.any(r) && hi % per && hi - hi % per >= lo) s.others(r, hi - hi % per + per, [&](bool) { ++others[r]; });
  }
  return s.job0 | static_cast<int64_t>(s.job1) << 32;
}
TWQ_TEST void twq_test_a16_plan(int64_t jobs, int64_t steps, const int* room, int per_sm, int warps, int all_there,
                                int64_t* out) {
  const twq::Plan p = twq::plan(jobs, steps, room, per_sm, warps, all_there != 0, 3);
  out[0] = p.clusters, out[1] = p.split_log, out[2] = p.parts;
}
