// rope.cu -- rotary positions of head rows, with the Q/K RMSNorm in the same pass.
//
// Each pair (x_a, x_b) of the first `rot` elements of a head row turns by its token's angle:
//   y_a = x_a cos - x_b sin,  y_b = x_b cos + x_a sin   (cos and sin times `factor`)
// where pair p is (2p, 2p + 1) (interleaved) or (p, p + rot/2) (halves).  With weights, x is
// first normalised: x * r * gamma * out_scale, r = 1 / sqrt(mean(x^2) + eps).  All in fp32,
// rounded once when stored.  The angle sum_a pos_a * freq_a is formed in 64 bits and reduced to
// a fraction of a turn before the fp32 sine and cosine: at position 10^6 a fp32 angle has lost
// all but a few bits of its fraction.  A block takes a few tokens, computes their cos/sin once
// into shared memory, and its warps then take the (token, head) rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "norm_math.cuh"
#include "rope.h"

namespace cpattn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store(float* p, float x) { *p = x; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// (cos, sin) * factor of pair p at position row `pr`.
__device__ __forceinline__ float2 pair_angle(const RopeCall& c, int pr, int p) {
  double turn = 0.0;
  for (int a = 0; a < c.n_axes; ++a)
    turn = fma(double(c.pos[(long long)pr * c.n_axes + a]), c.freq[(long long)a * (c.rot / 2) + p], turn);
  turn *= 0.15915494309189533577;  // 1 / (2 pi)
  turn -= rint(turn);
  float s, co;
  sincospif(2.0f * float(turn), &s, &co);
  return make_float2(co * c.factor, s * c.factor);
}

// One warp per head row, one element at a time: any D <= 256 and any even rot <= D.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_rows_kernel(const RopeCall c, int block_tokens) {
  extern __shared__ float2 cs[];  // [block_tokens][rot / 2]
  const int half = c.rot / 2, D = c.D;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int heads = 0;
  for (int t = 0; t < c.n_tensors; ++t) heads += c.t[t].heads;
  const int n_tiles = (c.tokens + block_tokens - 1) / block_tokens;
  for (int tile = blockIdx.x; tile < n_tiles; tile += gridDim.x) {
    const int t0 = tile * block_tokens;
    const int n_tok = min(block_tokens, c.tokens - t0);
    __syncthreads();  // the previous tile's angles are read no more
    for (int e = threadIdx.x; e < n_tok * half; e += kThreads)
      cs[e] = pair_angle(c, (t0 + e / half) % c.pos_rows, e % half);
    __syncthreads();
    for (int row = warp; row < n_tok * heads; row += kThreads / 32) {
      const int tk = row / heads;
      int h = row - tk * heads, ti = 0;
      while (h >= c.t[ti].heads) h -= c.t[ti++].heads;
      const RopeTensor& t = c.t[ti];
      const long long token = t0 + tk;
      const T* src = static_cast<const T*>(t.src) + token * t.src_stride + (long long)h * D;
      T* dst = static_cast<T*>(t.dst) + (h / t.group) * t.group_stride + token * t.dst_stride +
               (long long)(h % t.group) * D;
      if (t.gamma == nullptr && !t.rotate) {  // moved as it is, bit for bit
        for (int d = lane; d < D; d += 32) dst[d] = src[d];
        continue;
      }
      float x[kRopeMaxD / 32];
      // element index of this lane's value u: the rotated pairs' first and second elements in
      // turn, then the rest of the row
      auto index = [&](int u) {
        const int e = u * 32 + lane;  // position in the order a_0, b_0, a_1, b_1, ..., rest
        if (e >= c.rot || c.interleaved) return e;
        return (e & 1) ? (e >> 1) + half : (e >> 1);
      };
      float ss = 0.f;
#pragma unroll
      for (int u = 0; u < kRopeMaxD / 32; ++u) {
        x[u] = u * 32 + lane < D ? to_f32(src[index(u)]) : 0.f;
        ss = fmaf(x[u], x[u], ss);
      }
      if (t.gamma != nullptr) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float a = ss / float(D) + c.eps;
        const float r = a > 0.f ? rsqrt_refined(a) : 0.f;  // an all-zero row with eps = 0 stays 0
#pragma unroll
        for (int u = 0; u < kRopeMaxD / 32; ++u)
          if (u * 32 + lane < D) x[u] = x[u] * r * t.gamma[index(u)] * c.out_scale;
      }
      __syncwarp();  // in place: the whole row is read before any of it is written
#pragma unroll
      for (int u = 0; u < kRopeMaxD / 32; ++u) {
        const int e = u * 32 + lane;
        const float other = __shfl_xor_sync(0xffffffffu, x[u], 1);
        if (t.rotate && e < c.rot) {
          const float2 w = cs[tk * half + (e >> 1)];
          x[u] = (e & 1) ? fmaf(x[u], w.x, other * w.y) : fmaf(x[u], w.x, -other * w.y);
        }
        if (e < D) store(dst + index(u), x[u]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeCall& c, cudaStream_t stream) {
  const int block_tokens = 4;
  const int tiles = (c.tokens + block_tokens - 1) / block_tokens;
  const int cap = sm_count() * 8;
  const size_t smem = size_t(block_tokens) * (c.rot / 2) * sizeof(float2);
  const unsigned grid = unsigned(tiles < cap ? tiles : cap);
  if (c.f32) rope_rows_kernel<float><<<grid, kThreads, smem, stream>>>(c, block_tokens);
  else rope_rows_kernel<__nv_bfloat16><<<grid, kThreads, smem, stream>>>(c, block_tokens);
  return cudaGetLastError();
}

}  // namespace cpattn
