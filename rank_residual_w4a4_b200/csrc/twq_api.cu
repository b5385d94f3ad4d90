// C ABI of the library (include/twq.h): argument validation on the host, then
// stream-ordered launches. No entry point allocates device memory.
#include <string.h>

#include "twq_adapter.h"
#include "twq_internal.h"

namespace {

constexpr int kVersion = 100;  // 0.1.0

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

twq_status shape_ok(int64_t m, int64_t n, int64_t r) {
  if (m <= 0 || n <= 0 || r < 0) return TWQ_ERR_INVALID_ARG;
  if (m % 128 || n % 128) return TWQ_ERR_INVALID_ARG;
  if (r % 16) return TWQ_ERR_INVALID_ARG;
  if (r > 256) return TWQ_ERR_UNSUPPORTED;
  // TMA coordinates and element offsets are 32-bit in the kernels.
  if (m > (int64_t(1) << 24) || n > (int64_t(1) << 24)) return TWQ_ERR_UNSUPPORTED;
  return TWQ_OK;
}

twq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? TWQ_OK : TWQ_ERR_CUDA; }

// Checks shared by the three layer entry points. `need_res` / `need_lr` say
// which weight buffers the call reads.
twq_status check_layer(const uint8_t* xq, const float* sx, int64_t b, const twq_weights* w,
                       const void* y, bool need_res, bool need_lr) {
  if (!w) return TWQ_ERR_INVALID_ARG;
  twq_status s = shape_ok(w->m, w->n, w->r);
  if (s != TWQ_OK) return s;
  if (b < 0) return TWQ_ERR_INVALID_ARG;
  if (b > (int64_t(1) << 30)) return TWQ_ERR_UNSUPPORTED;
  if (b == 0) return TWQ_OK;
  if (!xq || !sx || !y) return TWQ_ERR_INVALID_ARG;
  if (!aligned16(xq) || !aligned16(sx) || !aligned16(y)) return TWQ_ERR_MISALIGNED;
  if (need_res) {
    if (!w->rq || !w->sr) return TWQ_ERR_INVALID_ARG;
    if (!aligned16(w->rq) || !aligned16(w->sr)) return TWQ_ERR_MISALIGNED;
  }
  if (need_lr) {
    if (w->r == 0) return TWQ_ERR_INVALID_ARG;
    if (!w->l1q || !w->sl1 || !w->l2t) return TWQ_ERR_INVALID_ARG;
    if (!aligned16(w->l1q) || !aligned16(w->sl1) || !aligned16(w->l2t)) return TWQ_ERR_MISALIGNED;
  }
  return TWQ_OK;
}

twq_status run(int mode, const uint8_t* xq, const float* sx, int64_t b, const twq_weights* w,
               void* out, const uint16_t* h, twq_stream_t stream) {
  twq::GemmCall c{mode, xq, sx, b, w, out, h};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (twq::decode_eligible(c)) return from_cuda(twq::launch_decode(c, st));
  return from_cuda(twq::launch_gemm(c, st, nullptr));
}

}  // namespace

extern "C" {

int twq_version(void) { return kVersion; }

const char* twq_status_string(twq_status s) {
  switch (s) {
    case TWQ_OK: return "ok";
    case TWQ_ERR_INVALID_ARG: return "invalid argument";
    case TWQ_ERR_UNSUPPORTED: return "unsupported shape";
    case TWQ_ERR_MISALIGNED: return "misaligned pointer or stride";
    case TWQ_ERR_CUDA: return "CUDA error";
    case TWQ_ERR_NOT_IMPLEMENTED: return "not implemented";
    case TWQ_ERR_DEVICE: return "device wait timed out";
  }
  return "unknown status";
}

twq_status twq_weights_sizes(int64_t m, int64_t n, int64_t r, size_t bytes_out[5]) {
  if (!bytes_out) return TWQ_ERR_INVALID_ARG;
  twq_status s = shape_ok(m, n, r);
  if (s != TWQ_OK) return s;
  const int64_t G = m / 128;
  bytes_out[0] = static_cast<size_t>(n * (m / 2));
  bytes_out[1] = static_cast<size_t>(G * n * 4);
  bytes_out[2] = static_cast<size_t>(r * (m / 2));
  bytes_out[3] = static_cast<size_t>(G * r * 4);
  bytes_out[4] = static_cast<size_t>(n * r * 2);
  return TWQ_OK;
}

twq_status twq_act_sizes(int64_t b, int64_t m, size_t bytes_out[2]) {
  if (!bytes_out || b < 0 || m <= 0 || m % 128) return TWQ_ERR_INVALID_ARG;
  if (m > (int64_t(1) << 24) || b > (int64_t(1) << 30)) return TWQ_ERR_UNSUPPORTED;
  bytes_out[0] = static_cast<size_t>(b * (m / 2));
  bytes_out[1] = static_cast<size_t>(b * (m / 128) * 4);
  return TWQ_OK;
}

twq_status twq_quantize_act(const uint16_t* x, int64_t b, int64_t m, int64_t ldx, uint8_t* xq,
                            float* sx, twq_stream_t stream) {
  if (b < 0 || m <= 0 || m % 128 || ldx < m) return TWQ_ERR_INVALID_ARG;
  if (m > (int64_t(1) << 24) || b > (int64_t(1) << 30)) return TWQ_ERR_UNSUPPORTED;
  if (b == 0) return TWQ_OK;
  if (!x || !xq || !sx) return TWQ_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(xq) || !aligned16(sx) || ldx % 8) return TWQ_ERR_MISALIGNED;
  return from_cuda(twq::launch_quantize_act(x, b, m, ldx, xq, sx,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

twq_status twq_quantize_act_a8(const uint16_t* x, int64_t b, int64_t m, int64_t ldx, int8_t* xq8,
                               float* sx, twq_stream_t stream) {
  if (b < 0 || m <= 0 || m % 128 || ldx < m) return TWQ_ERR_INVALID_ARG;
  if (m > (int64_t(1) << 24) || b > (int64_t(1) << 30)) return TWQ_ERR_UNSUPPORTED;
  if (b == 0) return TWQ_OK;
  if (!x || !xq8 || !sx) return TWQ_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(xq8) || !aligned16(sx) || ldx % 8) return TWQ_ERR_MISALIGNED;
  return from_cuda(twq::launch_quantize_act(x, b, m, ldx, reinterpret_cast<uint8_t*>(xq8), sx,
                                            reinterpret_cast<cudaStream_t>(stream), true));
}

twq_status twq_quantize_act_i8(const uint16_t* x, int64_t b, int64_t m, int64_t ldx, int8_t* xq8,
                               float* sx, twq_stream_t stream) {
  if (b < 0 || m <= 0 || m % 128 || ldx < m) return TWQ_ERR_INVALID_ARG;
  if (m > (int64_t(1) << 24) || b > (int64_t(1) << 30)) return TWQ_ERR_UNSUPPORTED;
  if (b == 0) return TWQ_OK;
  if (!x || !xq8 || !sx) return TWQ_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(xq8) || !aligned16(sx) || ldx % 8) return TWQ_ERR_MISALIGNED;
  return from_cuda(twq::launch_quantize_act(x, b, m, ldx, reinterpret_cast<uint8_t*>(xq8), sx,
                                            reinterpret_cast<cudaStream_t>(stream), false, true));
}

twq_status twq_pack_weights(const uint16_t* R, const uint16_t* L1, const uint16_t* L2,
                            const twq_weights* w, twq_stream_t stream) {
  if (!w) return TWQ_ERR_INVALID_ARG;
  twq_status s = shape_ok(w->m, w->n, w->r);
  if (s != TWQ_OK) return s;
  if (!R || !w->rq || !w->sr) return TWQ_ERR_INVALID_ARG;
  if (!aligned16(R) || !aligned16(w->rq) || !aligned16(w->sr)) return TWQ_ERR_MISALIGNED;
  if (w->r > 0) {
    if (!L1 || !L2 || !w->l1q || !w->sl1 || !w->l2t) return TWQ_ERR_INVALID_ARG;
    if (!aligned16(L1) || !aligned16(L2) || !aligned16(w->l1q) || !aligned16(w->sl1) ||
        !aligned16(w->l2t))
      return TWQ_ERR_MISALIGNED;
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = twq::launch_pack_cols(R, w->m, w->n, w->rq, w->sr, st);
  if (e == cudaSuccess && w->r > 0) e = twq::launch_pack_cols(L1, w->m, w->r, w->l1q, w->sl1, st);
  if (e == cudaSuccess && w->r > 0) e = twq::launch_transpose_bf16(L2, w->r, w->n, w->l2t, st);
  return from_cuda(e);
}

twq_status twq_fused_linear(const uint8_t* xq, const float* sx, int64_t b, const twq_weights* w,
                            uint16_t* y, twq_stream_t stream) {
  const bool lr = w && w->r > 0;
  twq_status s = check_layer(xq, sx, b, w, y, true, lr);
  if (s != TWQ_OK || b == 0) return s;
  return run(lr ? twq::kModeFused : twq::kModeW4A4, xq, sx, b, w, y, nullptr, stream);
}

twq_status twq_w4a4_only(const uint8_t* xq, const float* sx, int64_t b, const twq_weights* w,
                         uint16_t* y, twq_stream_t stream) {
  twq_status s = check_layer(xq, sx, b, w, y, true, false);
  if (s != TWQ_OK || b == 0) return s;
  return run(twq::kModeW4A4, xq, sx, b, w, y, nullptr, stream);
}

twq_status twq_lowrank_only(const uint8_t* xq, const float* sx, int64_t b, const twq_weights* w,
                            uint16_t* y, twq_stream_t stream) {
  twq_status s = check_layer(xq, sx, b, w, y, false, true);
  if (s != TWQ_OK || b == 0) return s;
  return run(twq::kModeLowRank, xq, sx, b, w, y, nullptr, stream);
}

twq_status twq_fused_linear_a8(const int8_t* xq8, const float* sx, int64_t b, const twq_weights* w,
                               uint16_t* y, twq_stream_t stream) {
  const bool lr = w && w->r > 0;
  const uint8_t* xq = reinterpret_cast<const uint8_t*>(xq8);
  twq_status s = check_layer(xq, sx, b, w, y, true, lr);
  if (s != TWQ_OK || b == 0) return s;
  twq::GemmCall c{lr ? twq::kModeFused : twq::kModeW4A4, xq, sx, b, w, y, nullptr};
  c.a8 = true;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (twq::decode_eligible(c)) return from_cuda(twq::launch_decode(c, st));
  return from_cuda(twq::launch_gemm(c, st, nullptr));
}

twq_status twq_fused_linear_i8(const int8_t* xq8, const float* sx, int64_t b, const twq_weights* w,
                               uint16_t* y, twq_stream_t stream) {
  return twq_fused_linear_a8(xq8, sx, b, w, y, stream);
}

twq_status twq_pack_l2_int4(const uint16_t* L2, int64_t r, int64_t n, uint8_t* l2q, float* sl2q,
                            twq_stream_t stream) {
  if (r <= 0 || r % 128 || n <= 0 || n % 128) return TWQ_ERR_INVALID_ARG;
  if (r > 256 || n > (int64_t(1) << 24)) return TWQ_ERR_UNSUPPORTED;
  if (!L2 || !l2q || !sl2q) return TWQ_ERR_INVALID_ARG;
  if (!aligned16(L2) || !aligned16(l2q) || !aligned16(sl2q)) return TWQ_ERR_MISALIGNED;
  return from_cuda(twq::launch_pack_cols(L2, r, n, l2q, sl2q, reinterpret_cast<cudaStream_t>(stream)));
}

twq_status twq_fused_linear_s2q(const uint8_t* xq, const float* sx, int64_t b, const twq_weights* w,
                                const uint8_t* l2q, const float* sl2q, uint16_t* y,
                                twq_stream_t stream) {
  if (!w) return TWQ_ERR_INVALID_ARG;
  if (w->r <= 0 || w->r % 128) return w->r > 0 ? TWQ_ERR_UNSUPPORTED : TWQ_ERR_INVALID_ARG;
  twq_status s = check_layer(xq, sx, b, w, y, true, false);
  if (s != TWQ_OK || b == 0) return s;
  if (!w->l1q || !w->sl1 || !l2q || !sl2q) return TWQ_ERR_INVALID_ARG;
  if (!aligned16(w->l1q) || !aligned16(w->sl1) || !aligned16(l2q) || !aligned16(sl2q))
    return TWQ_ERR_MISALIGNED;
  twq::GemmCall c{twq::kModeFusedS2Q, xq, sx, b, w, y, nullptr};
  c.l2q = l2q;
  c.sl2q = sl2q;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (twq::decode_eligible(c)) return from_cuda(twq::launch_decode(c, st));
  return from_cuda(twq::launch_gemm(c, st, nullptr));
}

// Validates a twq_fused_linear_x call (b >= 1) and fills the decode launch.
static twq_status prepare_fused_x(const uint16_t* x, int64_t ldx, int64_t b, const twq_weights* w,
                                  uint16_t* y, twq::GemmCall* out, bool a8 = false) {
  if (!x || !y || !w->rq || !w->sr) return TWQ_ERR_INVALID_ARG;
  if (!aligned16(x) || ldx % 8 || !aligned16(y) || !aligned16(w->rq) || !aligned16(w->sr))
    return TWQ_ERR_MISALIGNED;
  const bool lr = w->r > 0;
  if (lr) {
    if (!w->l1q || !w->sl1 || !w->l2t) return TWQ_ERR_INVALID_ARG;
    if (!aligned16(w->l1q) || !aligned16(w->sl1) || !aligned16(w->l2t)) return TWQ_ERR_MISALIGNED;
  }
  twq::GemmCall c{lr ? twq::kModeFused : twq::kModeW4A4, nullptr, nullptr, b, w, y, nullptr};
  c.x = x;
  c.ldx = ldx;
  c.a8 = a8;
  if (!twq::decode_eligible(c)) return TWQ_ERR_UNSUPPORTED;
  *out = c;
  return TWQ_OK;
}

twq_status twq_fused_linear_x(const uint16_t* x, int64_t ldx, int64_t b, const twq_weights* w,
                              uint16_t* y, twq_stream_t stream) {
  if (!w) return TWQ_ERR_INVALID_ARG;
  twq_status s = shape_ok(w->m, w->n, w->r);
  if (s != TWQ_OK) return s;
  if (b < 0 || ldx < w->m) return TWQ_ERR_INVALID_ARG;
  if (b == 0) return TWQ_OK;
  twq::GemmCall c{};
  if ((s = prepare_fused_x(x, ldx, b, w, y, &c)) != TWQ_OK) return s;
  return from_cuda(twq::launch_decode(c, reinterpret_cast<cudaStream_t>(stream)));
}

twq_status twq_fused_linear_x_a8(const uint16_t* x, int64_t ldx, int64_t b, const twq_weights* w,
                                 uint16_t* y, twq_stream_t stream) {
  if (!w) return TWQ_ERR_INVALID_ARG;
  twq_status s = shape_ok(w->m, w->n, w->r);
  if (s != TWQ_OK) return s;
  if (b < 0 || ldx < w->m) return TWQ_ERR_INVALID_ARG;
  if (b == 0) return TWQ_OK;
  twq::GemmCall c{};
  if ((s = prepare_fused_x(x, ldx, b, w, y, &c, true)) != TWQ_OK) return s;
  return from_cuda(twq::launch_decode(c, reinterpret_cast<cudaStream_t>(stream)));
}

twq_status twq_fused_linear_x_host(const uint16_t* x_host, int64_t b, const twq_weights* w,
                                   uint16_t* x_dev, uint16_t* y_dev, uint16_t* y_host,
                                   twq_stream_t stream) {
  if (!w) return TWQ_ERR_INVALID_ARG;
  twq_status s = shape_ok(w->m, w->n, w->r);
  if (s != TWQ_OK) return s;
  if (b < 0) return TWQ_ERR_INVALID_ARG;
  if (b == 0) return TWQ_OK;
  if (!x_host || !y_host) return TWQ_ERR_INVALID_ARG;
  twq::GemmCall c{};
  if ((s = prepare_fused_x(x_dev, w->m, b, w, y_dev, &c)) != TWQ_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t xb = static_cast<size_t>(b) * w->m * 2, yb = static_cast<size_t>(b) * w->n * 2;
  if (cudaMemcpyAsync(x_dev, x_host, xb, cudaMemcpyHostToDevice, st) != cudaSuccess)
    return TWQ_ERR_CUDA;
  cudaError_t e = twq::launch_decode(c, st);
  if (e != cudaSuccess) return from_cuda(e);
  if (cudaMemcpyAsync(y_host, y_dev, yb, cudaMemcpyDeviceToHost, st) != cudaSuccess)
    return TWQ_ERR_CUDA;
  return TWQ_OK;
}

twq_status twq_linear_host(const uint16_t* x_host, int64_t b, const twq_weights* w,
                           uint16_t* x_dev, int8_t* xq8, float* sx, uint16_t* y_dev,
                           uint16_t* y_host, twq_stream_t stream) {
  if (!w) return TWQ_ERR_INVALID_ARG;
  twq_status s = shape_ok(w->m, w->n, w->r);
  if (s != TWQ_OK) return s;
  if (b < 0) return TWQ_ERR_INVALID_ARG;
  if (b > (int64_t(1) << 30)) return TWQ_ERR_UNSUPPORTED;
  if (b == 0) return TWQ_OK;
  if (!x_host || !y_host || !x_dev || !y_dev) return TWQ_ERR_INVALID_ARG;
  if (!aligned16(x_dev)) return TWQ_ERR_MISALIGNED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t xb = static_cast<size_t>(b) * w->m * 2, yb = static_cast<size_t>(b) * w->n * 2;
  // Decode batches that the one-launch layer takes: no codes in HBM at all.
  twq::GemmCall c{};
  const bool one = prepare_fused_x(x_dev, w->m, b, w, y_dev, &c) == TWQ_OK;
  const uint8_t* xq = reinterpret_cast<const uint8_t*>(xq8);
  if (!one) {
    const bool lr = w->r > 0;
    if ((s = check_layer(xq, sx, b, w, y_dev, true, lr)) != TWQ_OK) return s;
  }
  if (cudaMemcpyAsync(x_dev, x_host, xb, cudaMemcpyHostToDevice, st) != cudaSuccess)
    return TWQ_ERR_CUDA;
  cudaError_t e;
  if (one) {
    e = twq::launch_decode(c, st);
  } else {
    // the codes one per byte (twq_quantize_act_i8), which the layer reads as they lie
    e = twq::launch_quantize_act(x_dev, b, w->m, w->m, reinterpret_cast<uint8_t*>(xq8), sx, st,
                                 false, true);
    if (e == cudaSuccess) {
      twq::GemmCall g{w->r > 0 ? twq::kModeFused : twq::kModeW4A4, xq, sx, b, w, y_dev, nullptr};
      g.a8 = true;
      e = twq::decode_eligible(g) ? twq::launch_decode(g, st) : twq::launch_gemm(g, st, nullptr);
    }
  }
  if (e != cudaSuccess) return from_cuda(e);
  if (cudaMemcpyAsync(y_host, y_dev, yb, cudaMemcpyDeviceToHost, st) != cudaSuccess)
    return TWQ_ERR_CUDA;
  return TWQ_OK;
}

size_t twq_unfused_workspace_bytes(int64_t b, int64_t n, int64_t r) {
  if (b <= 0 || n <= 0 || r < 0) return 0;
  // Y_res fp32 (b x n) | Y_lr fp32 (b x n) | H bf16 (b x r), each 256-byte aligned
  auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
  return up(size_t(b) * n * 4) * 2 + up(size_t(b) * r * 2);
}

twq_status twq_unfused_linear(const uint8_t* xq, const float* sx, int64_t b, const twq_weights* w,
                              uint16_t* y, void* workspace, size_t workspace_bytes,
                              twq_stream_t stream) {
  const bool lr = w && w->r > 0;
  twq_status s = check_layer(xq, sx, b, w, y, true, lr);
  if (s != TWQ_OK || b == 0) return s;
  if (!workspace) return TWQ_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return TWQ_ERR_MISALIGNED;
  if (workspace_bytes < twq_unfused_workspace_bytes(b, w->n, w->r)) return TWQ_ERR_INVALID_ARG;
  auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* yres = reinterpret_cast<float*>(ws);
  float* ylr = reinterpret_cast<float*>(ws + up(size_t(b) * w->n * 4));
  uint16_t* h = reinterpret_cast<uint16_t*>(ws + 2 * up(size_t(b) * w->n * 4));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!lr) return run(twq::kModeW4A4, xq, sx, b, w, y, nullptr, stream);
  s = run(twq::kModeResF32, xq, sx, b, w, yres, nullptr, stream);
  if (s == TWQ_OK) s = run(twq::kModeHOnly, xq, sx, b, w, h, nullptr, stream);
  if (s == TWQ_OK) s = run(twq::kModeS2F32, xq, sx, b, w, ylr, h, stream);
  if (s == TWQ_OK) s = from_cuda(twq::launch_add_cast(yres, ylr, b * w->n, y, st));
  return s;
}

namespace {

twq_status groups_ok(int64_t b, int64_t count) {
  if (b < 0 || count < 1) return TWQ_ERR_INVALID_ARG;
  if (b > twq::kMaxGroupRows || count > twq::kMaxGroups) return TWQ_ERR_UNSUPPORTED;
  return TWQ_OK;
}

twq_status adapter_shape_ok(int64_t m, int64_t n, int64_t r) {
  if (m <= 0 || n <= 0 || r <= 0 || m % 128 || n % 128 || r % 8) return TWQ_ERR_INVALID_ARG;
  if (r > 128 || m > (int64_t(1) << 20) || n > (int64_t(1) << 20)) return TWQ_ERR_UNSUPPORTED;
  return TWQ_OK;
}

// twq_selftest_adapter_stall: the calling thread's limit of the waits, or 0.
thread_local int64_t t_stall_ns = 0;

// Everything of an adapter call that does not depend on how X is stored.
twq_status check_adapters(int64_t b, const twq_adapters* ad, const twq_row_groups* g,
                          twq::AdapterCall* c) {
  if (!ad || !g) return TWQ_ERR_INVALID_ARG;
  twq_status s = adapter_shape_ok(ad->m, ad->n, ad->r);
  if (s == TWQ_OK) s = groups_ok(b, ad->count);
  if (s != TWQ_OK) return s;
  if (g->b != b || g->count != ad->count) return TWQ_ERR_INVALID_ARG;
  if (!ad->a || !ad->b || !ad->scale) return TWQ_ERR_INVALID_ARG;
  // twq_group_rows' own rule: an empty batch has no order
  if ((b > 0 && !g->order) || !g->offsets || !g->tiles) return TWQ_ERR_INVALID_ARG;
  if (!aligned16(ad->a) || !aligned16(ad->b) || !aligned16(ad->scale) || !aligned16(g->order) ||
      !aligned16(g->offsets) || !aligned16(g->tiles))
    return TWQ_ERR_MISALIGNED;
  *c = twq::AdapterCall{};
  c->g = twq::RowGroupsView{static_cast<int>(b), static_cast<int>(ad->count), g->order, g->offsets,
                            reinterpret_cast<int4*>(g->tiles)};
  c->m = static_cast<int>(ad->m);
  c->n = static_cast<int>(ad->n);
  c->r = static_cast<int>(ad->r);
  c->a = ad->a;
  c->bm = ad->b;
  c->scale = ad->scale;
  c->wait_ns = t_stall_ns ? static_cast<uint64_t>(t_stall_ns) : twq::kAdapterWaitNs;
  c->stall = t_stall_ns != 0;
  return TWQ_OK;
}

twq_status set_x(twq::AdapterCall* c, const uint16_t* x, int64_t ldx) {
  if (!x || ldx < c->m) return TWQ_ERR_INVALID_ARG;
  if (!aligned16(x) || ldx % 8) return TWQ_ERR_MISALIGNED;
  c->x = x;
  c->ldx = ldx;
  return TWQ_OK;
}

twq_status set_codes(twq::AdapterCall* c, const int8_t* xq8, const float* sx) {
  if (!xq8 || !sx) return TWQ_ERR_INVALID_ARG;
  if (!aligned16(xq8) || !aligned16(sx)) return TWQ_ERR_MISALIGNED;
  c->xq8 = xq8;
  c->sx = sx;
  return TWQ_OK;
}

twq_status run_linear(twq::AdapterCall* c, const uint16_t* base, uint16_t* h, uint16_t* y,
                      twq_stream_t stream) {
  if (!h || !y) return TWQ_ERR_INVALID_ARG;
  if (!aligned16(base) || !aligned16(h) || !aligned16(y)) return TWQ_ERR_MISALIGNED;
  c->base = base;
  c->h = h;
  c->y = y;
  return from_cuda(twq::launch_adapter_linear(*c, reinterpret_cast<cudaStream_t>(stream)));
}

twq_status run_backward(twq::AdapterCall* c, const uint16_t* dy, const uint16_t* h,
                        const uint16_t* dx_base, uint16_t* dx, uint16_t* da, uint16_t* db,
                        void* workspace, size_t workspace_bytes, twq_stream_t stream) {
  if (c->g.b > 0) {
    if (!dy || !h || !dx) return TWQ_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(h) || !aligned16(dx) || !aligned16(dx_base))
      return TWQ_ERR_MISALIGNED;
  }
  const size_t need =
      twq_adapter_backward_workspace_bytes(c->g.b, c->m, c->n, c->r, c->g.count);
  if (!da || !db || (need && !workspace)) return TWQ_ERR_INVALID_ARG;
  if (!aligned16(da) || !aligned16(db) || !aligned16(workspace)) return TWQ_ERR_MISALIGNED;
  if (workspace_bytes < need) return TWQ_ERR_INVALID_ARG;
  c->dy = dy;
  c->h = const_cast<uint16_t*>(h);  // read only in the backward pass
  c->base = dx_base;
  c->dx = dx;
  c->da = da;
  c->db = db;
  c->workspace = workspace;
  return from_cuda(twq::launch_adapter_backward(*c, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

twq_status twq_row_groups_sizes(int64_t b, int64_t count, size_t bytes_out[3]) {
  if (!bytes_out) return TWQ_ERR_INVALID_ARG;
  const twq_status s = groups_ok(b, count);
  if (s != TWQ_OK) return s;
  bytes_out[0] = static_cast<size_t>(b) * 4;
  bytes_out[1] = static_cast<size_t>(count + 1) * 4;
  bytes_out[2] = 16 * (1 + static_cast<size_t>(twq::small_tiles_cap(b, count)) +
                       static_cast<size_t>(twq::row_tiles_cap(b, count, 128))) +
                 4 * static_cast<size_t>(count + 1);
  return TWQ_OK;
}

twq_status twq_group_rows(const int32_t* ids, const twq_row_groups* g, twq_stream_t stream) {
  if (!g) return TWQ_ERR_INVALID_ARG;
  const twq_status s = groups_ok(g->b, g->count);
  if (s != TWQ_OK) return s;
  if (!g->offsets || !g->tiles || (g->b > 0 && (!ids || !g->order))) return TWQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(ids) % 4 || !aligned16(g->order) || !aligned16(g->offsets) ||
      !aligned16(g->tiles))
    return TWQ_ERR_MISALIGNED;
  const twq::RowGroupsView v{static_cast<int>(g->b), static_cast<int>(g->count), g->order,
                             g->offsets, reinterpret_cast<int4*>(g->tiles)};
  return from_cuda(twq::launch_group_rows(ids, v, reinterpret_cast<cudaStream_t>(stream)));
}

twq_status twq_adapter_linear(const uint16_t* x, int64_t ldx, int64_t b, const twq_adapters* ad,
                              const twq_row_groups* g, const uint16_t* base, uint16_t* h,
                              uint16_t* y, twq_stream_t stream) {
  twq::AdapterCall c;
  twq_status s = check_adapters(b, ad, g, &c);
  if (s != TWQ_OK || b == 0) return s;
  s = set_x(&c, x, ldx);
  return s != TWQ_OK ? s : run_linear(&c, base, h, y, stream);
}

twq_status twq_adapter_linear_i8(const int8_t* xq8, const float* sx, int64_t b,
                                 const twq_adapters* ad, const twq_row_groups* g,
                                 const uint16_t* base, uint16_t* h, uint16_t* y,
                                 twq_stream_t stream) {
  twq::AdapterCall c;
  twq_status s = check_adapters(b, ad, g, &c);
  if (s != TWQ_OK || b == 0) return s;
  s = set_codes(&c, xq8, sx);
  return s != TWQ_OK ? s : run_linear(&c, base, h, y, stream);
}

size_t twq_adapter_backward_workspace_bytes(int64_t b, int64_t m, int64_t n, int64_t r,
                                            int64_t count) {
  if (groups_ok(b, count) != TWQ_OK || adapter_shape_ok(m, n, r) != TWQ_OK) return 0;
  return twq::adapter_backward_workspace(b, m, n, r, count);
}

twq_status twq_adapter_backward(const uint16_t* dy, const uint16_t* x, int64_t ldx,
                                const uint16_t* h, int64_t b, const twq_adapters* ad,
                                const twq_row_groups* g, const uint16_t* dx_base, uint16_t* dx,
                                uint16_t* da, uint16_t* db, void* workspace,
                                size_t workspace_bytes, twq_stream_t stream) {
  twq::AdapterCall c;
  twq_status s = check_adapters(b, ad, g, &c);
  if (s == TWQ_OK && b > 0) s = set_x(&c, x, ldx);
  return s != TWQ_OK ? s
                     : run_backward(&c, dy, h, dx_base, dx, da, db, workspace, workspace_bytes,
                                    stream);
}

twq_status twq_adapter_backward_i8(const uint16_t* dy, const int8_t* xq8, const float* sx,
                                   const uint16_t* h, int64_t b, const twq_adapters* ad,
                                   const twq_row_groups* g, const uint16_t* dx_base, uint16_t* dx,
                                   uint16_t* da, uint16_t* db, void* workspace,
                                   size_t workspace_bytes, twq_stream_t stream) {
  twq::AdapterCall c;
  twq_status s = check_adapters(b, ad, g, &c);
  if (s == TWQ_OK && b > 0) s = set_codes(&c, xq8, sx);
  return s != TWQ_OK ? s
                     : run_backward(&c, dy, h, dx_base, dx, da, db, workspace, workspace_bytes,
                                    stream);
}

twq_status twq_device_status(int* code) {
  if (!code) return TWQ_ERR_INVALID_ARG;
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return TWQ_ERR_CUDA;
  int c1 = 0, c2 = 0, c3 = 0, c4 = 0;
  e = twq::read_and_clear_device_status(&c1);
  if (e == cudaSuccess) e = twq::read_and_clear_decode_status(&c2);
  if (e == cudaSuccess) e = twq::read_and_clear_pair_status(&c3);
  if (e == cudaSuccess) e = twq::read_and_clear_adapter_status(&c4);
  if (e != cudaSuccess) return TWQ_ERR_CUDA;
  *code = c1 ? c1 : (c2 ? c2 : (c3 ? c3 : c4));
  return *code ? TWQ_ERR_DEVICE : TWQ_OK;
}

twq_status twq_selftest_wait_timeout(const uint8_t* xq, const float* sx, int64_t b,
                                     const twq_weights* w, uint16_t* y, int64_t wait_limit_ns,
                                     twq_stream_t stream) {
  twq_status s = check_layer(xq, sx, b, w, y, true, false);
  if (s != TWQ_OK) return s;
  if (wait_limit_ns < 1000 || wait_limit_ns > 1000000000) return TWQ_ERR_INVALID_ARG;
  twq::GemmCall c{twq::kModeW4A4, xq, sx, b, w, y, nullptr};
  if (!twq::pair_eligible(c)) return TWQ_ERR_UNSUPPORTED;
  return from_cuda(twq::launch_pair_stall_selftest(c, reinterpret_cast<cudaStream_t>(stream),
                                                   static_cast<unsigned long long>(wait_limit_ns)));
}

twq_status twq_selftest_adapter_stall(int64_t wait_limit_ns) {
  if (wait_limit_ns != 0 && (wait_limit_ns < 1000 || wait_limit_ns > 1000000000)) return TWQ_ERR_INVALID_ARG;
  t_stall_ns = wait_limit_ns;
  return TWQ_OK;
}

void twq_release_cache(void) {
  twq::release_decode_cache();
  twq::release_noalloc_cache();
  twq::release_adapter_cache();
}

int twq_launches_per_call(const char* ep) {
  if (!ep) return -1;
  if (!strcmp(ep, "twq_quantize_act") || !strcmp(ep, "twq_quantize_act_a8")) return 1;
  if (!strcmp(ep, "twq_pack_weights")) return 3;
  if (!strcmp(ep, "twq_pack_l2_int4") || !strcmp(ep, "twq_fused_linear_s2q")) return 1;
  if (!strcmp(ep, "twq_fused_linear") || !strcmp(ep, "twq_w4a4_only") ||
      !strcmp(ep, "twq_lowrank_only") || !strcmp(ep, "twq_fused_linear_x") ||
      !strcmp(ep, "twq_fused_linear_x_host") || !strcmp(ep, "twq_fused_linear_a8") ||
      !strcmp(ep, "twq_fused_linear_x_a8") || !strcmp(ep, "twq_quantize_act_i8") ||
      !strcmp(ep, "twq_fused_linear_i8"))
    return 1;
  if (!strcmp(ep, "twq_linear_host")) return 2;
  if (!strcmp(ep, "twq_selftest_wait_timeout")) return 1;  // 1 for the batches twq_fused_linear_x takes
  if (!strcmp(ep, "twq_unfused_linear") || !strcmp(ep, "twq_unfused_linear_noalloc")) return 4;
  if (!strcmp(ep, "twq_fold_transforms")) return 5;
  if (!strcmp(ep, "twq_group_rows")) return 1;
  if (!strcmp(ep, "twq_adapter_linear") || !strcmp(ep, "twq_adapter_linear_i8")) return 2;
  if (!strcmp(ep, "twq_adapter_backward") || !strcmp(ep, "twq_adapter_backward_i8")) return 5;
  return -1;
}

}  // extern "C"
