// window_rows.cu -- windowed attention with one warp per query row, on the CUDA cores.
//
// For query row (b, i, h) at position p the warp walks the row's visible keys -- the early
// (sink) keys [0, early), then the window [lo, hi) -- with an online softmax in fp32:
//   m' = max(m, s), l' = l e^(m - m') + e^(s - m'), acc' = acc e^(m - m') + e^(s - m') v.
// Hidden keys are never read.  Lane l holds elements d = l, l + 32, ... of q and of the
// accumulator.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sm100_ptx.cuh"
#include "window.h"

namespace cpattn {
namespace {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename In, int T>
__global__ void __launch_bounds__(256) window_rows_kernel(const WindowCall c) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= (long long)c.B * c.Sq * c.H) return;
  const int h = int(row % c.H);  // (b, i, h), h fastest
  const int i = int((row / c.H) % c.Sq);
  const int b = int(row / ((long long)c.H * c.Sq));
  const int kvh = h / (c.H / c.Hkv);
  const int len = sequence_length(c, b);
  const int p = (c.from_end ? len - c.Sq : c.off) + i;
  const KeyRange r = visible_keys(p, c.left, c.right, c.sinks, len);
  const In* qp = static_cast<const In*>(c.q) + ((long long)b * c.Sq + i) * c.q_stride + (long long)h * c.D;
  const In* kp = static_cast<const In*>(c.k) + (long long)b * c.Skv * c.k_stride + (long long)kvh * c.D;
  const In* vp = static_cast<const In*>(c.v) + (long long)b * c.Skv * c.v_stride + (long long)kvh * c.D;
  float qv[T], acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int d = lane + 32 * t;
    qv[t] = d < c.D ? to_f32(qp[d]) : 0.f;
    acc[t] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int n = r.early + (r.hi - r.lo);
  for (int e = 0; e < n; ++e) {
    const int j = e < r.early ? e : r.lo + (e - r.early);
    float part = 0.f;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int d = lane + 32 * t;
      if (d < c.D) part = fmaf(qv[t], to_f32(kp[j * c.k_stride + d]), part);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    const float s = part * c.scale;
    if (s > m) {
      const float corr = expf(m - s);
      l *= corr;
#pragma unroll
      for (int t = 0; t < T; ++t) acc[t] *= corr;
      m = s;
    }
    const float w = expf(s - m);
    l += w;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int d = lane + 32 * t;
      if (d < c.D) acc[t] = fmaf(w, to_f32(vp[j * c.v_stride + d]), acc[t]);
    }
  }
  const long long o_off = row * c.D;
  const long long li = ((long long)b * c.H + h) * c.Sq + i;
  float wo = n > 0 ? 1.0f / l : 0.f;  // no visible key: O = 0, LSE = -inf
  float L = n > 0 ? m + logf(l) : -INFINITY, wa = 0.f;
  if (c.accumulate) {
    if (n == 0) return;  // nothing to add: the running row stays as it is
    const float la = c.lse[li];
    const float mx = fmaxf(la, L);
    const float ea = expf(la - mx), ec = expf(L - mx);
    wa = ea / (ea + ec);
    wo *= ec / (ea + ec);
    L = mx + logf(ea + ec);
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int d = lane + 32 * t;
    if (d >= c.D) continue;
    float o = acc[t] * wo;
    if (c.out_f32) {
      float* dst = static_cast<float*>(c.out) + o_off + d;
      if (wa != 0.f) o = fmaf(wa, *dst, o);  // an empty accumulator row is not read
      *dst = o;
    } else {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(c.out) + o_off + d;
      if (wa != 0.f) o = fmaf(wa, __bfloat162float(*dst), o);
      *dst = __float2bfloat16_rn(o);
    }
  }
  __syncwarp();  // every lane's read of the running LSE precedes lane 0's write
  if (lane == 0 && c.lse != nullptr) c.lse[li] = L;
}

template <typename In>
cudaError_t launch(const WindowCall& c, cudaStream_t stream) {
  const long long blocks = ((long long)c.B * c.Sq * c.H + 7) / 8;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned g = unsigned(blocks);
  if (c.D <= 64) window_rows_kernel<In, 2><<<g, 256, 0, stream>>>(c);
  else if (c.D <= 128) window_rows_kernel<In, 4><<<g, 256, 0, stream>>>(c);
  else window_rows_kernel<In, 8><<<g, 256, 0, stream>>>(c);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_rows(const WindowCall& c, cudaStream_t stream) {
  return c.in_f32 ? launch<float>(c, stream) : launch<__nv_bfloat16>(c, stream);
}

}  // namespace cpattn
