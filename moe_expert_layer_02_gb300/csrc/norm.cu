// norm.cu -- the residual's addition and the root-mean-square norm in front of
// the layer, with rows quantised for the experts, and the gradient.
//
//   h = x + r;  m = rsqrt(mean(h^2) + eps);  y = h m gamma
//   s = max|y| / 448 (1 where that is zero);  q = e4m3(y / s)
// with u = gamma dy and dh the gradient that arrives on h itself:
//   dx = dr = m u - h m^3 mean(u h) + dh
//   dgamma = sum_t dy_t h_t m_t
// (the pre-norm of a transformer block; "Optimising Ling-2.6-1T on TPU with
// SGLang-JAX", s.5 activation quantisation; "Kimi K3 on the Google TPU
// ecosystem: feasibility analysis", s.2.4 RMSNorm.)
//
// The norm is taken from the fp32 sum x + r, so y and q are rounded once, from
// that; the stored h is its rounding to the caller's type.  Both passes are bound by
// memory; on GB300, against the 6764 GB/s of a plain copy, 16384 x 8192 bf16 with
// residual and fp8 rows takes 178 us (6.8 TB/s), the gradient of 8192 x 7168 bf16
// 74 us (6.4 TB/s; its second kernel, the sum of the blocks' dgamma, 3 of them).
#include <algorithm>

#include "device.cuh"
#include "internal.h"
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kNormThreads = 256;

// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float block_sum(float v, float* s_red) {
  v = warp_sum(v);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
  if (lane == 0) s_red[warp] = v;
  __syncthreads();
  v = lane < n ? s_red[lane] : 0.0f;
  v = warp_sum(v);
  __syncthreads();
  return v;
}

__device__ __forceinline__ float block_max(float v, float* s_red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
  if (lane == 0) s_red[warp] = v;
  __syncthreads();
  v = lane < n ? s_red[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  return v;
}

// Scale of a quantised row: 1 for a row of zeros, and for one whose scale rounds to
// zero; a NaN stays one.
__device__ __forceinline__ float row_scale(float amax) {
  const float s = amax / 448.0f;
  return s == 0.0f ? 1.0f : s;
}

// y / s as near as e4m3's rounding needs it: z has the code of the quotient rounded to
// fp32.  p = y * (1 / s), both rounded, is within two units of its last place of that, so
// it serves wherever no midpoint between two codes lies as near: those have the low 20
// bits 0x80000 from 2^-6 on (and below it, where the steps stay those of 2^-6, once 2^-6
// is added).  Values within kNear units of one are divided, with the others of their
// vector (one vector of 30000), and so are rows whose 1 / s is no normal number.
// 16384 x 8192 bf16 177.0 us, 1216 rows 18.5, 8 rows 3.32; everything divided 179.5, 19.7
// and 3.60; p alone, which misses one code in a million, 176.8, 18.3 and 3.24.
struct QuantBy {
  float s, inv;
  __device__ __forceinline__ explicit QuantBy(float scale)
      : s(scale), inv(scale >= 0x1p-120f ? 1.0f / scale : 0.0f) {}
  template <int V>
  __device__ __forceinline__ void operator()(const float (&y)[V], float (&z)[V]) const {
    constexpr uint32_t kNear = 4;
    uint32_t low = ~0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      z[i] = y[i] * inv;
      float u = fabsf(z[i]);
      if (u < 0x1p-6f) u += 0x1p-6f;  // the steps below 2^-6 are those above it
      // how far above the midpoint less kNear, in the upper 20 bits
      low = min(low, (__float_as_uint(u) << 12) + ((0x80000u + kNear) << 12));
    }
    if (low <= (2 * kNear) << 12 || inv == 0.0f) {
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] = y[i] / s;
    }
  }
};

// V codes of consecutive values, in words of up to four.
template <int V>
__device__ __forceinline__ void store_codes(uint8_t* q, const float (&y)[V], const QuantBy& by) {
  if constexpr (V == 1) {
    float z[1];
    by(y, z);
    *q = f32_to_e4m3(z[0]);
  } else {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float four[4] = {y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]};
      float z[4];
      by(four, z);
      const uint32_t lo =
          __nv_cvt_float2_to_fp8x2(make_float2(z[0], z[1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi =
          __nv_cvt_float2_to_fp8x2(make_float2(z[2], z[3]), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    }
    if constexpr (V == 8)
      *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(q) = w[0];
  }
}

template <typename E, int V>
__device__ __forceinline__ void load_sum(const E* x, const E* r, size_t at, float (&h)[V]) {
  using RV = RowVec<E, V>;
  using Raw = typename RV::Raw;
  RV::unpack(reinterpret_cast<const Raw*>(x)[at], h);
  if (r) {
    float b[V];
    RV::unpack(reinterpret_cast<const Raw*>(r)[at], b);
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] += b[i];
  }
}

// Sum (or NaN-keeping maximum) over the warps of one row: tpr threads, a
// multiple of 32; a block holds whole rows, and all of its threads call this.
// s_red has one word per warp.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, int tpr, float* s_red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? max_nan(v, w) : v + w;
  }
  if (tpr == 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = tpr >> 5;
  if (lane == 0) s_red[warp] = v;
  __syncthreads();
  v = lane < nw ? s_red[warp / nw * nw + lane] : 0.0f;  // 0 is the neutral element of both
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? max_nan(v, w) : v + w;
  }
  return v;
}

// A row stays in registers: tpr threads hold NV vectors each, blockDim / tpr
// rows per block.  Of a shifted row these are the vectors that lie inside it (and
// whose gamma lies inside two whole vectors of gamma); the `head` elements before
// them and the `tail` after them, fewer than 3 V <= 24, are one each of the first
// threads.  h_out and y_out may be x and r: a thread writes what it has read alone.
template <typename E, int V, int NV, int THREADS, bool SHIFTED>
__global__ void __launch_bounds__(THREADS)
    add_rmsnorm_kernel(const E* x, const E* r, const E* __restrict__ gamma, E* h_out, E* y_out,
                       uint8_t* __restrict__ q, float* __restrict__ q_scale, int T, int H, int tpr,
                       float eps) {
  pdl_wait();
  pdl_release();
  using RV = RowVec<E, V>;
  using Raw = typename RV::Raw;
  __shared__ float s_sum[32], s_max[32];
  const int group = threadIdx.x / tpr, me = threadIdx.x - group * tpr;
  const size_t t = (size_t)blockIdx.x * (blockDim.x / tpr) + group;
  const bool live = t < (size_t)T;
  int head = 0, n = H / V, col = -1;  // col: the thread's element outside the vectors
  if constexpr (SHIFTED) {
    head = min(H, (int)((V - t * H % V) % V));
    n = (H - head) / V;
    if (head > 0 && n > 0 && (n + 1) * V > H) --n;
    const int tail = H - head - n * V;
    if (live) col = me < head ? me : me < head + tail ? H - tail + me - head : -1;
  }
  const size_t first = (t * H + head) / V, at = t * H + col;
  Raw a[NV], b[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = me + j * tpr;
    if (live && v < n) {
      a[j] = __ldcs(reinterpret_cast<const Raw*>(x) + first + v);
      if (r) b[j] = __ldcs(reinterpret_cast<const Raw*>(r) + first + v);
    }
  }
  float h[NV][V], one = 0.0f;
  if (SHIFTED && col >= 0) {
    one = widen(x[at]);
    if (r) one += widen(r[at]);
    if (h_out) h_out[at] = narrow<E>(one);
  }
  float sq = one * one;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = me + j * tpr;
    if (live && v < n) {
      RV::unpack(a[j], h[j]);
      if (r) {
        float f[V];
        RV::unpack(b[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i) h[j][i] += f[i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) sq = fmaf(h[j][i], h[j][i], sq);
      if (h_out) reinterpret_cast<Raw*>(h_out)[first + v] = RV::pack(h[j]);
    }
  }
  const float m = rsqrtf(row_reduce<false>(sq, tpr, s_sum) / (float)H + eps);
  float amax = 0.0f;
  if (SHIFTED && col >= 0) {
    one = one * m * widen(gamma[col]);
    amax = max_nan(amax, fabsf(one));
    if (y_out) y_out[at] = narrow<E>(one);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = me + j * tpr;
    if (live && v < n) {
      const Raw* gv = reinterpret_cast<const Raw*>(gamma) + v;
      Raw raw = __ldg(gv);
      if constexpr (SHIFTED)
        if (head) raw = take16<sizeof(E)>(raw, __ldg(gv + 1), head * (int)sizeof(E));
      float g[V];
      RV::unpack(raw, g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        h[j][i] = h[j][i] * m * g[i];
        amax = max_nan(amax, fabsf(h[j][i]));
      }
      if (y_out) reinterpret_cast<Raw*>(y_out)[first + v] = RV::pack(h[j]);
    }
  }
  if (!q) return;
  const float s = row_scale(row_reduce<true>(amax, tpr, s_max));
  if (live && me == 0) q_scale[t] = s;
  const QuantBy by(s);
  if (SHIFTED && col >= 0) q[at] = f32_to_e4m3(one / s);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = me + j * tpr;
    if (live && v < n) store_codes<V>(q + (first + v) * V, h[j], by);
  }
}

// One block per row; the row is read again for each of its passes.  h_out and y_out may
// be x and r, so they are written in the last one, by the thread that read the element
// (1024 x 65536 bf16 191 us; 181 with h written in the first and y in the second pass).
template <typename E, int V>
__global__ void __launch_bounds__(kNormThreads)
    add_rmsnorm_loop_kernel(const E* x, const E* r, const E* __restrict__ gamma, E* h_out,
                            E* y_out, uint8_t* __restrict__ q, float* __restrict__ q_scale, int H,
                            float eps) {
  pdl_wait();
  pdl_release();
  using RV = RowVec<E, V>;
  using Raw = typename RV::Raw;
  __shared__ float s_red[32];
  const int n = H / V;
  const size_t t = blockIdx.x;
  float sq = 0.0f;
  for (int v = threadIdx.x; v < n; v += blockDim.x) {
    float h[V];
    load_sum<E, V>(x, r, t * n + v, h);
#pragma unroll
    for (int i = 0; i < V; ++i) sq = fmaf(h[i], h[i], sq);
  }
  const float m = rsqrtf(block_sum(sq, s_red) / (float)H + eps);
  // one vector of y in place of h, both stored if this is the last pass
  auto norm = [&](int v, float (&h)[V], bool last) {
    float g[V];
    load_sum<E, V>(x, r, t * n + v, h);
    if (last && h_out) reinterpret_cast<Raw*>(h_out)[t * n + v] = RV::pack(h);
    RV::unpack(reinterpret_cast<const Raw*>(gamma)[v], g);
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = h[i] * m * g[i];
    if (last && y_out) reinterpret_cast<Raw*>(y_out)[t * n + v] = RV::pack(h);
  };
  float s = 1.0f;
  if (q) {
    float amax = 0.0f;
    for (int v = threadIdx.x; v < n; v += blockDim.x) {
      float y[V];
      norm(v, y, false);
#pragma unroll
      for (int i = 0; i < V; ++i) amax = max_nan(amax, fabsf(y[i]));
    }
    s = row_scale(block_max(amax, s_red));
    if (threadIdx.x == 0) q_scale[t] = s;
  }
  const QuantBy by(s);
  for (int v = threadIdx.x; v < n; v += blockDim.x) {
    float y[V];
    norm(v, y, true);
    if (q) store_codes<V>(q + t * H + (size_t)v * V, y, by);
  }
}

// Blocks take rows b, b + grid, ...; each keeps its own sum of dgamma over its
// rows in its row of `part` [grid][H], in row order.
template <typename E, int V>
__global__ void __launch_bounds__(kNormThreads)
    add_rmsnorm_backward_loop_kernel(const E* __restrict__ h_in, const E* __restrict__ gamma,
                                     const E* __restrict__ dy, const E* __restrict__ dh,
                                     E* __restrict__ dx, float* __restrict__ part, int T, int H,
                                     float eps) {
  pdl_wait();
  pdl_release();
  using RV = RowVec<E, V>;
  using Raw = typename RV::Raw;
  __shared__ float s_red[32];
  const int n = H / V;
  float* mine = part ? part + (size_t)blockIdx.x * H : nullptr;
  for (size_t t = blockIdx.x; t < (size_t)T; t += gridDim.x) {
    float sq = 0.0f, dot = 0.0f;
    for (int v = threadIdx.x; v < n; v += blockDim.x) {
      float h[V], g[V], d[V];
      RV::unpack(reinterpret_cast<const Raw*>(h_in)[t * n + v], h);
      RV::unpack(reinterpret_cast<const Raw*>(gamma)[v], g);
      RV::unpack(reinterpret_cast<const Raw*>(dy)[t * n + v], d);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sq = fmaf(h[i], h[i], sq);
        dot = fmaf(h[i] * g[i], d[i], dot);
      }
    }
    const float m = rsqrtf(block_sum(sq, s_red) / (float)H + eps);
    const float c = block_sum(dot, s_red) * m * m / (float)H;
    for (int v = threadIdx.x; v < n; v += blockDim.x) {
      float h[V], g[V], d[V], o[V];
      RV::unpack(reinterpret_cast<const Raw*>(h_in)[t * n + v], h);
      RV::unpack(reinterpret_cast<const Raw*>(gamma)[v], g);
      RV::unpack(reinterpret_cast<const Raw*>(dy)[t * n + v], d);
      float b[V];
#pragma unroll
      for (int i = 0; i < V; ++i) b[i] = 0.0f;
      if (dh) RV::unpack(reinterpret_cast<const Raw*>(dh)[t * n + v], b);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // every product and sum spelled out: the compiler's choice of fused ones
        // would make dx depend on which other outputs are asked for
        o[i] = fmaf(m, fmaf(-h[i], c, g[i] * d[i]), b[i]);
        if (mine) {
          const size_t col = (size_t)v * V + i;
          mine[col] = fmaf(d[i], h[i] * m, t == blockIdx.x ? 0.0f : mine[col]);
        }
      }
      reinterpret_cast<Raw*>(dx)[t * n + v] = RV::pack(o);
    }
  }
}

// Sums of two values over a warp at once: lanes 0-15 get a's, lanes 16-31 b's.
__device__ __forceinline__ float warp_sum_two(float a, float b) {
  const bool low = (threadIdx.x & 16) == 0;
  float v = low ? a : b;
  v += __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The gradient with a row in registers: tpr threads (a multiple of 32, at most
// 512) hold NV vectors each, a block's blockDim / tpr row groups go through the
// rows together, and a thread's columns stay the same, so its sums of dgamma stay
// in registers as well.  (With SHIFTED they do because a group's rows are a multiple
// of V apart.)  Instructions bound it once memory does not: packed fp32 arithmetic
// and one reduction for both sums took 8192 x 7168 bf16 from 110 to 76 us.  The
// vectors of the STAGES - 1 next rows are on their way into
// shared memory (each thread copies and reads its own: no barrier) while this one is
// reduced.  The groups' sums of dgamma are added in group order into the block's
// row of `part`; with CLUSTER the grid is one cluster, whose blocks add each other's
// sums up in shared memory, in block order, into dgamma itself.
template <typename E, int V, int NV, int STAGES, bool SHIFTED, bool CLUSTER>
__global__ void __launch_bounds__(512, 1)
    add_rmsnorm_backward_kernel(const E* __restrict__ h_in, const E* __restrict__ gamma,
                                const E* __restrict__ dy, const E* __restrict__ dh,
                                E* __restrict__ dx, float* __restrict__ part, int T, int H,
                                int tpr, float eps) {
  pdl_wait();
  pdl_release();
  using RV = RowVec<E, V>;
  using Raw = typename RV::Raw;
  using FV = FloatVec<V>;
  extern __shared__ uint4 s_dyn[];
  Raw* ring = reinterpret_cast<Raw*>(s_dyn);  // [STAGES][3 or 2][NV][blockDim]
  __shared__ float s_red[2][2][16];
  const int group = threadIdx.x / tpr, me = threadIdx.x - group * tpr;
  const int groups = blockDim.x / tpr, step = gridDim.x * groups;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = tpr >> 5;
  const int stage_len = (dh ? 3 : 2) * NV * blockDim.x;  // vectors
  const float inv_h = 1.0f / (float)H;
  // a block's groups walk side by side: the same number of steps for all of them
  const int64_t base0 = (int64_t)blockIdx.x * groups;
  const size_t t0 = (size_t)base0 + group;
  const int shift = SHIFTED ? (int)(t0 * H % V) : 0, n = (H + shift + V - 1) / V;
  auto lo = [&](int v) { return SHIFTED && v == 0 ? shift : 0; };
  auto hi = [&](int v) { return SHIFTED ? min(V, H + shift - v * V) : V; };
  auto whole = [&](int v) { return !SHIFTED || (lo(v) == 0 && hi(v) == V); };
  FV acc[NV];
  // gamma stays in registers while they last; the widest rows read it again (L1)
  constexpr bool kKeep = NV * sizeof(Raw) <= 32;
  auto load_gamma = [&](int v) {
    if constexpr (SHIFTED) return load_part<E, V>(gamma + v * V - shift, lo(v), hi(v));
    return __ldg(reinterpret_cast<const Raw*>(gamma) + v);
  };
  Raw g[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (kKeep && me + j * tpr < n) g[j] = load_gamma(me + j * tpr);
    acc[j] = FV::splat(0.0f);
  }
  auto gamma_of = [&](int j) {
    return vload<E, V>(kKeep ? g[j] : load_gamma(me + j * tpr));
  };
  const size_t row0 = (t0 * H - shift) / V + me;
  const size_t hop = (size_t)step * H / V;  // SHIFTED: step is a multiple of V, or not taken
  size_t next = row0;  // the thread's first vector of the next row to fetch
  Raw* xp = reinterpret_cast<Raw*>(dx) + row0;
  // copies the next row that has not been fetched yet into stage `stage`
  auto fetch = [&](int64_t t, int stage) {
    if (t < T) {
      Raw* to = ring + stage * stage_len + threadIdx.x;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int v = me + j * tpr;
        if (v < n) {
          const size_t at = next + j * tpr;
          const Raw* hp = reinterpret_cast<const Raw*>(h_in) + at;
          const Raw* dp = reinterpret_cast<const Raw*>(dy) + at;
          const Raw* bp = reinterpret_cast<const Raw*>(dh) + at;
          if constexpr (SHIFTED) {
            // the operand may end inside its last vector
            const int bytes = (int)min((size_t)V, (size_t)T * H - at * V) * (int)sizeof(E);
            copy_async_part(to + j * blockDim.x, hp, bytes);
            copy_async_part(to + (NV + j) * blockDim.x, dp, bytes);
            if (dh) copy_async_part(to + (2 * NV + j) * blockDim.x, bp, bytes);
          } else {
            copy_async(to + j * blockDim.x, hp);
            copy_async(to + (NV + j) * blockDim.x, dp);
            if (dh) copy_async(to + (2 * NV + j) * blockDim.x, bp);
          }
        }
      }
      next += hop;
    }
    copy_async_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch((int64_t)t0 + (int64_t)i * step, i);
  int stage = 0, flip = 0;
  for (int64_t base = base0; base < T; base += step) {
    const int64_t t = base + group;
    const bool live = t < T;
    const Raw* from = ring + stage * stage_len + threadIdx.x;
    fetch(t + (int64_t)(STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
    copy_async_wait<STAGES - 1>();
    FV h[NV], d[NV], sq = FV::splat(0.0f), dot = FV::splat(0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = me + j * tpr;
      if (live && v < n) {
        Raw hr = from[j * blockDim.x], dr = from[(NV + j) * blockDim.x];
        if (!whole(v)) {
          hr = keep_part<E, V>(hr, lo(v), hi(v));
          dr = keep_part<E, V>(dr, lo(v), hi(v));
        }
        h[j] = vload<E, V>(hr);
        d[j] = vload<E, V>(dr);
        sq = vfma(h[j], h[j], sq);
        dot = vfma(vmul(h[j], gamma_of(j)), d[j], dot);
      }
    }
    // sums of squares in the lower lanes, of products in the upper ones
    float two = warp_sum_two(sq.sum(), dot.sum());
    if (tpr > 32) {
      // two buffers in turn: a step's one barrier also keeps the next step's
      // writes behind this one's reads
      if ((lane & 15) == 0) s_red[flip][lane >> 4][warp] = two;
      __syncthreads();
      two = (lane & 15) < nw ? s_red[flip][lane >> 4][warp / nw * nw + (lane & 15)] : 0.0f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) two += __shfl_xor_sync(0xffffffffu, two, o);
      flip ^= 1;
    }
    const float m = rsqrtf(__shfl_sync(0xffffffffu, two, 0) * inv_h + eps);
    const FV c = FV::splat(-(__shfl_sync(0xffffffffu, two, 16) * inv_h) * m * m);
    const FV mv = FV::splat(m);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = me + j * tpr;
      if (live && v < n) {
        FV b = FV::splat(0.0f);
        if (dh) b = vload<E, V>(from[(2 * NV + j) * blockDim.x]);
        // m (gamma dy - h c) + dh
        const FV o = vfma(mv, vfma(h[j], c, vmul(gamma_of(j), d[j])), b);
        const FV add = vfma(d[j], vmul(h[j], mv), acc[j]);
        if (whole(v)) {
          xp[j * tpr] = vpack<E, V>(o);
        } else {
          store_part<E, V>(reinterpret_cast<E*>(xp + j * tpr), vpack<E, V>(o), lo(v), hi(v));
        }
        acc[j] = add;
      }
    }
    xp += hop;
    if (++stage == STAGES) stage = 0;
  }
  if (!part) return;
  // in place of the ring: the groups' sums [groups][H], then the block's [H]
  float* s_acc = reinterpret_cast<float*>(s_dyn);
  float* s_sum = groups > 1 ? s_acc + groups * H : s_acc;
  copy_async_wait<0>();  // past the last step's wait only empty groups are left
  __syncthreads();
  // through shared memory even for one group: eight floats a lane apart, stores of one
  // float each to global memory take 4 us
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = me + j * tpr;
    if (v >= n) continue;
    float* mine = s_acc + group * H + v * V - shift;
    float f[V];
    acc[j].get(f);
    if constexpr (SHIFTED) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i >= lo(v) && i < hi(v)) mine[i] = f[i];
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4)
        *reinterpret_cast<float4*>(mine + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    }
  }
  __syncthreads();
  // four columns at a time, for their loads to overlap
  const bool spread = CLUSTER && gridDim.x > 1;
  for (int c0 = threadIdx.x; c0 < H; c0 += 4 * blockDim.x) {
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = 0; k < groups; ++k)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        sum[u] += s_acc[k * H + min(c0 + u * (int)blockDim.x, H - 1)];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + u * blockDim.x;
      if (c < H) (spread ? s_sum : part + (size_t)blockIdx.x * H)[c] = sum[u];
    }
  }
  if constexpr (CLUSTER) {
    if (!spread) return;
    cluster_sync();
    const int blocks = gridDim.x, hop = blocks * blockDim.x;
    for (int c = blockIdx.x * blockDim.x + threadIdx.x; c < H; c += hop) {
      float v[kMaxCluster], sum = 0.0f;
#pragma unroll
      for (int b = 0; b < kMaxCluster; ++b)
        v[b] = b < blocks ? __uint_as_float(load_cluster(mapa_shared(smem_u32(s_sum + c), b)))
                          : 0.0f;
#pragma unroll
      for (int b = 0; b < kMaxCluster; ++b) sum += v[b];
      part[c] = sum;
    }
    cluster_sync();  // no block leaves while another reads its sums
  }
}

// dgamma[c] = sum_g part[g][c]: 32 columns a block, eight warps that take
// every eighth row and whose sums are added in warp order.
__global__ void __launch_bounds__(kNormThreads)
    column_sum_kernel(const float* __restrict__ part, float* __restrict__ out, int G, int H) {
  pdl_wait();
  pdl_release();
  __shared__ float s_sum[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float acc = 0.0f;
  if (c < H) {
#pragma unroll 8
    for (int g = warp; g < G; g += 8) acc += part[(size_t)g * H + c];
  }
  s_sum[warp][lane] = acc;
  __syncthreads();
  if (warp == 0 && c < H) {
#pragma unroll
    for (int w = 1; w < 8; ++w) acc += s_sum[w][lane];
    out[c] = acc;
  }
}

// Blocks of the gradient: one a multiprocessor, in eights (a shifted row's place in
// its vectors repeats every V rows at the latest), one row each at least.
int norm_backward_blocks(int T) {
  const int sms = device_sm_count();
  return std::min(T, sms < 8 ? 8 : sms / 8 * 8);
}

int round32(int v) { return (v + 31) / 32 * 32; }

}  // namespace

size_t norm_workspace_bytes(int T, int H) {
  return (size_t)norm_backward_blocks(T) * H * sizeof(float) + 256;
}

cudaError_t launch_add_rmsnorm(const void* x, const void* r, const void* gamma, void* h, void* y,
                               void* q, float* q_scale, int T, int H, int dtype, float eps,
                               cudaStream_t s) {
  const int eb = dtype_bytes(dtype);
  RowPath path = row_path((size_t)H * eb, x, r, gamma, h, y);
  if (reinterpret_cast<uintptr_t>(q) % (16 / eb)) path = kScalar;  // a vector's codes are one store
  return by_row_path(dtype, path, [&](auto elem, auto width, auto way) {
    using E = decltype(elem);
    constexpr int V = decltype(width)::value;
    constexpr bool kShift = decltype(way)::value == kShifted;
    constexpr int kMany = V == 1 ? 8 : 4;  // vectors a thread, for rows in registers
    const int n = std::max(1, H / V);
    auto go = [&](auto kern, int threads, int tpr) {
      const int rows = threads / tpr;
      count_launch();
      return launch_kernel(kern, dim3((unsigned)(((int64_t)T + rows - 1) / rows)),
                           dim3(rows * tpr), 0, s, 1,
                           static_cast<const E*>(x), static_cast<const E*>(r),
                           static_cast<const E*>(gamma), static_cast<E*>(h), static_cast<E*>(y),
                           static_cast<uint8_t*>(q), q_scale, T, H, tpr, eps);
    };
    // few rows: one vector a thread, for the shortest way through a row, while a
    // multiprocessor's 1024 of them hold all rows (8192 bf16 with codes, against four: 64
    // rows 3.5 and 4.1 us, 152 rows 3.7 and 4.3, 160 rows 5.4 and 4.7, 304 rows 5.4 and 5.1,
    // 608 rows 12.3 and 9.7; 304 x 2880 2.9 and 4.0)
    const int one = round32(n), sms = device_sm_count();
    if (n <= 1024 && T <= 2 * sms && T * one <= 1024 * sms)
      return go(add_rmsnorm_kernel<E, V, 1, 1024, kShift>, one, one);
    const int tpr = round32((n + kMany - 1) / kMany);
    if (tpr <= 256) return go(add_rmsnorm_kernel<E, V, kMany, 256, kShift>, 256, tpr);
    if (tpr <= 1024) return go(add_rmsnorm_kernel<E, V, kMany, 1024, kShift>, tpr, tpr);
    constexpr int kLoopV = kShift ? 1 : V;
    count_launch();
    return launch_kernel(add_rmsnorm_loop_kernel<E, kLoopV>, dim3(T), dim3(kNormThreads), 0, s, 1,
                         static_cast<const E*>(x), static_cast<const E*>(r),
                         static_cast<const E*>(gamma), static_cast<E*>(h), static_cast<E*>(y),
                         static_cast<uint8_t*>(q), q_scale, H, eps);
  });
}

cudaError_t launch_add_rmsnorm_backward(const void* h, const void* gamma, const void* dy,
                                        const void* dh, void* dx, float* dgamma, void* ws, int T,
                                        int H, int dtype, float eps, cudaStream_t s) {
  float* part = dgamma ? static_cast<float*>(ws) : nullptr;
  const RowPath path = row_path((size_t)H * dtype_bytes(dtype), h, gamma, dy, dh, dx);
  int G = norm_backward_blocks(T);
  bool summed = false;  // dgamma written by the first kernel
  cudaError_t e = by_row_path(dtype, path, [&](auto elem, auto width, auto way) {
    using E = decltype(elem);
    constexpr int V = decltype(width)::value;
    constexpr bool kShift = decltype(way)::value == kShifted;
    if constexpr (V > 1) {
      const int n = kShift ? (H + 2 * V - 2) / V : H / V;  // vectors of a row, at most
      auto go = [&](auto nv_, auto stages_) {
        constexpr int nv = decltype(nv_)::value, stages = decltype(stages_)::value;
        const int tpr = round32((n + nv - 1) / nv), groups = 512 / tpr, block = groups * tpr;
        const int one_step = (int)(((int64_t)T + groups - 1) / groups);
        const int G_ = std::min(G, one_step);
        const int64_t steps = ((int64_t)one_step + G_ - 1) / G_;
        // as many stages of the ring as a block has rows
        size_t smem = (size_t)std::min<int64_t>(stages, steps) * (dh ? 3 : 2) * nv * block * 16;
        smem = std::max(smem, (size_t)(groups > 1 ? groups + 1 : 1) * H * sizeof(float));
        constexpr int kSmem = 192 * 1024;  // any ring at its widest row
        auto run = [&](auto kern, cudaError_t ready, int cluster, float* sums) {
          if (ready != cudaSuccess) return ready;
          count_launch();
          return launch_kernel(kern, dim3(G), dim3(block), smem, s, cluster,
                               static_cast<const E*>(h), static_cast<const E*>(gamma),
                               static_cast<const E*>(dy), static_cast<const E*>(dh),
                               static_cast<E*>(dx), sums, T, H, tpr, eps);
        };
        if (dgamma && one_step <= kMaxCluster) {
          // one cluster of up to eight blocks, a power of two (blocks without a row add
          // nothing), saves the sum's own launch: one row of 8192 bf16 3.7 us on the GPU
          // and 6.6 a call, 4.8 and 8.4 with it; eight rows 5.5 and 6.9, 5.1 and 8.6
          for (G = 1; G < one_step;) G *= 2;
          summed = true;
          constexpr auto kern = add_rmsnorm_backward_kernel<E, V, nv, stages, kShift, true>;
          return run(kern, ensure_max_smem<kern>(kSmem), G, dgamma);
        }
        G = G_;  // fewer than a multiple of eight only for a single step
        constexpr auto kern = add_rmsnorm_backward_kernel<E, V, nv, stages, kShift, false>;
        return run(kern, ensure_max_smem<kern>(kSmem), 1, part);
      };
      using Two = std::integral_constant<int, 2>;
      using Four = std::integral_constant<int, 4>;
      // two vectors a thread and a ring of four rows; four and two where a row needs it
      // (for a narrower one slower: 4000 x 4096 fp32 43.7 and 46.1 us)
      if (n <= 1024) return go(Two{}, Four{});
      if (n <= 2048) return go(Four{}, Two{});
    }
    constexpr int kLoopV = kShift ? 1 : V;
    count_launch();
    return launch_kernel(add_rmsnorm_backward_loop_kernel<E, kLoopV>, dim3(G), dim3(kNormThreads),
                         0, s, 1, static_cast<const E*>(h), static_cast<const E*>(gamma),
                         static_cast<const E*>(dy), static_cast<const E*>(dh),
                         static_cast<E*>(dx), part, T, H, eps);
  });
  if (e != cudaSuccess || !dgamma || summed) return e;
  count_launch();
  return launch_kernel(column_sum_kernel, dim3((H + 31) / 32), dim3(kNormThreads), 0, s, 1,
                       static_cast<const float*>(part), dgamma, G, H);
}

}  // namespace moe
