// window_f32.cu -- windowed attention and its single-token form with fp32 inputs, on the CUDA cores.
//
// A block takes 32 or 64 query rows of one (b, h) and walks the keys that some row of them sees --
// early (sink) keys, then the window, as one list -- 64 at a time: S = Q K^T, the online softmax in
// base 2 and O += P V, all in fp32 (fp32 has no tensor-core product that keeps its digits).  Keys
// of the list that a row does not see weigh exactly 0; keys outside the list are never read.
// Thread (ty, tx) of 16 x 16 holds R rows from R ty on, of S the keys tx + 16 j and of O the columns
// 4 tx + 64 g: an inner step of four columns is R + 4 16-byte reads for 16 R FMAs.  The FMA pipe
// and the shared-memory port bound it about equally (26 TFLOP/s at 3000 x 8 heads of 128).  Rows are
// padded by 4 floats, so the 16 keys of a read fall in different banks.  D is padded to 64, 128 or
// 256 with zeros.  K and V have one buffer each and still arrive behind the arithmetic: the next K
// is copied during the softmax and P V, the next V during the next S.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "api_common.h"
#include "kernels.h"
#include "sm100_ptx.cuh"
#include "window.h"

namespace cpattn {
namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 64;
constexpr float kLn2 = 0.69314718055994530942f;

template <int kBytes>
__device__ __forceinline__ void cp_async(float* dst, const float* src, bool live) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 4 : 0)
                 : "memory");
}

// R rows a thread, 16 R a block.
template <int DP, int R>
struct Tile {
  static constexpr int kRows = 16 * R;
  static constexpr int kStride = DP + 4;
  static constexpr int kOffK = kRows * kStride;
  static constexpr int kOffV = kOffK + kKeys * kStride;
  static constexpr int kOffP = kOffV + kKeys * kStride;
  static constexpr int kSmem = (kOffP + kRows * (kKeys + 4)) * 4;
};

template <int DP, int R>
__global__ void __launch_bounds__(kThreads, 2) window_f32_kernel(const __grid_constant__ WindowCall c, int n_tiles,
                                                              float scale_log2, bool vec) {
  using T = Tile<DP, R>;
  constexpr int kG = DP / 64, kRows = T::kRows;
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;
  float* sk = sm + T::kOffK;
  float* sv = sm + T::kOffV;
  float* sp = sm + T::kOffP;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int tile = n_tiles - 1 - int(blockIdx.x % unsigned(n_tiles));
  const int bh = int(blockIdx.x / unsigned(n_tiles));
  const int b = bh / c.H, h = bh - b * c.H, kvh = h / (c.H / c.Hkv);
  const int q0 = tile * kRows, n_rows = min(kRows, c.Sq - q0);

  griddep_wait();
  griddep_release();

  const int len = sequence_length(c, b);
  const int off = c.from_end ? len - c.Sq : c.off;
  int early, lo, n;  // keys that some row sees: [0, early), then [lo, lo + n - early)
  {
    const KeyRange a = visible_keys(off + q0, c.left, c.right, c.sinks, len);
    const KeyRange z = visible_keys(off + q0 + n_rows - 1, c.left, c.right, c.sinks, len);
    lo = a.lo < z.hi ? a.lo : z.hi;
    early = c.sinks < lo ? c.sinks : lo;
    n = early + (z.hi - lo);
  }
  const float* qp = static_cast<const float*>(c.q) + ((long long)b * c.Sq + q0) * c.q_stride + (long long)h * c.D;
  const float* kp = static_cast<const float*>(c.k) + (long long)b * c.Skv * c.k_stride + (long long)kvh * c.D;
  const float* vp = static_cast<const float*>(c.v) + (long long)b * c.Skv * c.v_stride + (long long)kvh * c.D;

  // copy rows 0 .. n_live - 1 of `dst` from token row(r) in the background, zeros elsewhere: one
  // cp.async group, of 16 bytes where every row allows it, else of 4
  auto fetch = [&](float* dst, int rows, int n_live, const float* base, long long stride, auto row) {
    if (vec) {
      for (int e = threadIdx.x; e < rows * (DP / 4); e += kThreads) {
        const int r = e / (DP / 4), d = 4 * (e % (DP / 4));
        const bool live = r < n_live && d < c.D;
        cp_async<16>(dst + r * T::kStride + d, live ? base + row(r) * stride + d : base, live);
      }
    } else {
      for (int e = threadIdx.x; e < rows * DP; e += kThreads) {
        const int r = e / DP, d = e % DP;
        const bool live = r < n_live && d < c.D;
        cp_async<4>(dst + r * T::kStride + d, live ? base + row(r) * stride + d : base, live);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto key_at = [&](int e) { return (long long)(e < early ? e : lo + (e - early)); };
  auto fetch_keys = [&](float* dst, const float* base, long long stride, int e0) {
    fetch(dst, kKeys, min(kKeys, n - e0), base, stride, [&](int r) { return key_at(e0 + r); });
  };
  fetch(sq, kRows, n_rows, qp, c.q_stride, [](int r) { return (long long)r; });
  if (n > 0) {
    fetch_keys(sk, kp, c.k_stride, 0);
    fetch_keys(sv, vp, c.v_stride, 0);
  }

  KeyRange see[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    see[i] = visible_keys(off + q0 + min(R * ty + i, n_rows - 1), c.left, c.right, c.sinks, len);
  float m[R], l[R];
  float4 o[R][kG];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int g = 0; g < kG; ++g) o[i][g] = make_float4(0.f, 0.f, 0.f, 0.f);
  }

  for (int e0 = 0; e0 < n; e0 += kKeys) {
    const int live = min(kKeys, n - e0);
    const bool more = e0 + kKeys < n;
    asm volatile("cp.async.wait_group 1;" ::: "memory");  // Q and these keys; their values may be under way
    __syncthreads();
    float s[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 8
    for (int d = 0; d < DP; d += 4) {
      float4 q[R], k[4];
#pragma unroll
      for (int i = 0; i < R; ++i) q[i] = *reinterpret_cast<const float4*>(sq + (R * ty + i) * T::kStride + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * T::kStride + d);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = fmaf(q[i].x, k[j].x, s[i][j]);
          s[i][j] = fmaf(q[i].y, k[j].y, s[i][j]);
          s[i][j] = fmaf(q[i].z, k[j].z, s[i][j]);
          s[i][j] = fmaf(q[i].w, k[j].w, s[i][j]);
        }
    }
    __syncthreads();  // K is read: the next keys' may come, while the softmax and P V run
    if (more) fetch_keys(sk, kp, c.k_stride, e0 + kKeys);
    else asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = tx + 16 * j;
        const int key = int(key_at(e0 + r));
        const bool seen = r < live && key < see[i].hi && (key >= see[i].lo || key < see[i].early);
        s[i][j] = seen ? s[i][j] * scale_log2 : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      if (mx > m[i]) {  // the same for the row's 16 threads
        const float a = ex2(m[i] - mx);
        m[i] = mx;
        l[i] *= a;
#pragma unroll
        for (int g = 0; g < kG; ++g) o[i][g].x *= a, o[i][g].y *= a, o[i][g].z *= a, o[i][g].w *= a;
      }
      const float ref = m[i] == -INFINITY ? 0.f : m[i];  // no key seen so far: every weight is 0
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = ex2(s[i][j] - ref);
        l[i] += p;
        sp[(R * ty + i) * (kKeys + 4) + tx + 16 * j] = p;
      }
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");  // the values
    __syncthreads();  // (a row's weights are written and read by one half-warp)
#pragma unroll 4
    for (int j = 0; j < kKeys; j += 4) {
      float4 p[R];
#pragma unroll
      for (int i = 0; i < R; ++i) p[i] = *reinterpret_cast<const float4*>(sp + (R * ty + i) * (kKeys + 4) + j);
#pragma unroll
      for (int g = 0; g < kG; ++g) {
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const float4 v = *reinterpret_cast<const float4*>(sv + (j + jj) * T::kStride + 4 * tx + 64 * g);
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const float w = jj == 0 ? p[i].x : jj == 1 ? p[i].y : jj == 2 ? p[i].z : p[i].w;
            o[i][g].x = fmaf(w, v.x, o[i][g].x);
            o[i][g].y = fmaf(w, v.y, o[i][g].y);
            o[i][g].z = fmaf(w, v.z, o[i][g].z);
            o[i][g].w = fmaf(w, v.w, o[i][g].w);
          }
        }
      }
    }
    if (more) {
      __syncthreads();  // V is read: the next one's copy runs beside the next S
      fetch_keys(sv, vp, c.v_stride, e0 + kKeys);
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");

#pragma unroll
  for (int i = 0; i < R; ++i) {
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
    const int r = R * ty + i;
    if (r >= n_rows) continue;
    const bool empty = m[i] == -INFINITY;  // no visible key: O = 0, LSE = -inf
    const float inv = empty ? 0.f : 1.0f / l[i];
    const long long at = (((long long)b * c.Sq + q0 + r) * c.H + h) * c.D;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const float f[4] = {o[i][g].x * inv, o[i][g].y * inv, o[i][g].z * inv, o[i][g].w * inv};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int d = 4 * tx + 64 * g + x;
        if (d >= c.D) continue;
        if (c.out_f32) static_cast<float*>(c.out)[at + d] = f[x];
        else static_cast<__nv_bfloat16*>(c.out)[at + d] = __float2bfloat16_rn(f[x]);
      }
    }
    if (tx == 0 && c.lse != nullptr)
      c.lse[((long long)b * c.H + h) * c.Sq + q0 + r] = empty ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
  }
}

template <int DP, int R>
cudaError_t launch(const WindowCall& c, cudaStream_t stream) {
  static SmemOptIn opt_in;
  cudaError_t e = opt_in(reinterpret_cast<const void*>(window_f32_kernel<DP, R>), Tile<DP, R>::kSmem);
  if (e != cudaSuccess) return e;
  const int n_tiles = (c.Sq + 16 * R - 1) / (16 * R);
  const bool vec = c.D % 4 == 0 && c.q_stride % 4 == 0 && c.k_stride % 4 == 0 && c.v_stride % 4 == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(n_tiles) * c.H * c.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Tile<DP, R>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, window_f32_kernel<DP, R>, c, n_tiles,
                            float(double(c.scale) * 1.4426950408889634074), vec);
}

// Four rows a thread read shared memory half as often for their products; two give twice the
// blocks, for calls whose 64-row blocks would leave SMs idle.  Measured: 3000 x 8 heads of 128, 384
// blocks of 64 rows, 417 us against 475; 1000 x 4 heads of 64, 64 of them, 35 against 25.  At
// D = 256 four rows do not fit the registers of two blocks per SM.
template <int DP>
cudaError_t launch_rows(const WindowCall& c, cudaStream_t stream) {
  const long long blocks = (long long)((c.Sq + 63) / 64) * c.H * c.B;
  if constexpr (DP <= 128)
    if (blocks >= 2LL * sm_count()) return launch<DP, 4>(c, stream);
  return launch<DP, 2>(c, stream);
}

}  // namespace

cudaError_t launch_window_f32(const WindowCall& c, cudaStream_t stream) {
  if (c.D <= 64) return launch_rows<64>(c, stream);
  if (c.D <= 128) return launch_rows<128>(c, stream);
  return launch_rows<256>(c, stream);
}

}  // namespace cpattn
