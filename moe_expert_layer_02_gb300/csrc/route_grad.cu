// route_grad.cu -- gradient of the routing weights with respect to the logits.
//
// Softmax over the chosen logits: w_j = exp(l_j) / sum_i exp(l_i), so with
// d_j = dL/dw_j
//   dL/dl_j = w_j (d_j - c),  c = sum_i w_i d_i.
// Renormalised sigmoid scores: w_j = s_j / S, s_j = sigmoid(l_j), S = sum_i s_i,
//   dL/dl_j = s_j (1 - s_j) (d_j - c) / S.
// Logits that were not chosen get zero.  ("Kimi K3 on the Google TPU ecosystem:
// feasibility analysis", s.2.4 moe_renormalize; "Optimising Ling-2.6-1T on TPU
// with SGLang-JAX", s.1 top-8 routing.)  The dense rows that are written bound it: on
// GB300, 16384 x 256 top-8 4.2 us (16.8 MB written and 1.6 read: 4.4 TB/s with launch and
// start), 4096 x 896 top-16 with sigmoid 4.0 us (14.7 and 1.0 MB: 3.9 TB/s).
#include "device.cuh"
#include "internal.h"
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kRouteWarps = 8;

// One warp per token, lane j holding slot j.  The token's row of the gradient
// is put together in shared memory (slots of one expert add up in slot order)
// and written once, zeros included.
template <bool SIGMOID>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_backward_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                          const float* __restrict__ w, const float* __restrict__ dw,
                          float* __restrict__ dlogits, int T, int E, int k, int* err) {
  pdl_wait();
  pdl_release();
  extern __shared__ __align__(16) float s_rows[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t t = (size_t)blockIdx.x * kRouteWarps + warp;
  if (t >= (size_t)T) return;
  float* row = s_rows + warp * E;
  for (int i = lane; i < E; i += 32) row[i] = 0.0f;
  int e = -1;
  if (lane < k) {
    e = idx[t * k + lane];
    if ((unsigned)e >= (unsigned)E) {
      if (e != -1) record_error(err, kErrInvalidArg);
      e = -1;
    }
  }
  const float wj = e >= 0 ? w[t * k + lane] : 0.0f;
  const float dj = e >= 0 ? dw[t * k + lane] : 0.0f;
  float d = dj - warp_sum(wj * dj);
  if (SIGMOID) {
    // s and s (1 - s) from exp(-|l|), which neither overflows nor cancels
    const float l = e >= 0 ? logits[t * E + e] : 0.0f;
    const float x = expf(-fabsf(l)), r = 1.0f / (1.0f + x);
    const float score = e >= 0 ? (l >= 0.0f ? r : x * r) : 0.0f;
    const float total = warp_sum(score);
    // a NaN stays one; scores that have all underflowed have no gradient
    d = total == 0.0f ? 0.0f : x * r * r * d / total;
  } else {
    d *= wj;
  }
  __syncwarp();
  // slots of one expert, if there are any (a lane finds another's mark in place of
  // its own), add up in slot order
  if (e >= 0) row[e] = __int_as_float(lane);
  __syncwarp();
  const bool alone = e < 0 || __float_as_int(row[e]) == lane;
  if (__all_sync(0xffffffffu, alone)) {
    if (e >= 0) row[e] = d;
  } else {
    if (e >= 0) row[e] = 0.0f;
    __syncwarp();
    for (int j = 0; j < k; ++j) {
      if (lane == j && e >= 0) row[e] += d;
      __syncwarp();
    }
  }
  __syncwarp();
  if (E % 4 == 0 && reinterpret_cast<uintptr_t>(dlogits) % 16 == 0) {
    for (int i = lane; i < E / 4; i += 32)
      reinterpret_cast<float4*>(dlogits + t * E)[i] = reinterpret_cast<const float4*>(row)[i];
  } else {
    for (int i = lane; i < E; i += 32) dlogits[t * E + i] = row[i];
  }
}

}  // namespace

cudaError_t launch_route_backward(const float* logits, const int32_t* idx, const float* w,
                                  const float* dw, float* dlogits, int sigmoid, int T, int E,
                                  int k, int* err, cudaStream_t s) {
  const dim3 grid((T + kRouteWarps - 1) / kRouteWarps), block(kRouteWarps * 32);
  const size_t smem = (size_t)kRouteWarps * E * sizeof(float);
  count_launch();
  if (sigmoid)
    return launch_kernel(route_backward_kernel<true>, grid, block, smem, s, 1, logits, idx, w, dw,
                         dlogits, T, E, k, err);
  return launch_kernel(route_backward_kernel<false>, grid, block, smem, s, 1, logits, idx, w, dw,
                       dlogits, T, E, k, err);
}

}  // namespace moe
