// Test harness: exposes the host's division of a launch on BF16 activations to the CPU tests. It
// compiles the kernel's own translation unit, so the plan under test is the one the library makes;
// only host code runs (no device, no launch).
#include "twq_a16_sm100.cu"

// room: 4 numbers of clusters; out: clusters, log2 of their blocks, parts, steps of a block at most.
extern "C" __attribute__((visibility("default"))) int twq_test_a16_plan(int64_t jobs, int64_t steps, const int* room,
                                                                        int per_sm, int warps, int all_there, int most,
                                                                        int64_t* out) {
  if (jobs < 1 || steps < 1 || !room || per_sm < 1 || warps < 1 || most < 0 || most > 3 || !out) return 1;
  const twq::Plan p = twq::plan(jobs, steps, room, per_sm, warps, all_there != 0, most);
  out[0] = p.clusters, out[1] = p.split_log, out[2] = p.parts, out[3] = p.mine;
  return 0;
}
