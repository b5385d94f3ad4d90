// Test harness: exposes what the host computes for launches on BF16 activations to the CPU tests. It
// compiles the kernel's own translation unit; only host code runs (no device, no launch).
#include "twq_a16_sm100.cu"

#define TWQ_TEST extern "C" __attribute__((visibility("default")))

// Limits of a block's waits and of its wait for peers' parts, in ns.
TWQ_TEST uint64_t twq_test_a16_wait_limit(uint64_t ns, int stall, int rank) {
  return twq::wait_limit(ns, stall != 0, rank);
}
TWQ_TEST uint64_t twq_test_a16_parts_limit(uint64_t ns, int stall, int split, int steps) {
  return twq::parts_limit(ns, stall != 0, split, steps);
}
