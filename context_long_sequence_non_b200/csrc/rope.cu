// rope.cu -- rotary positions of head rows, with the Q/K RMSNorm in the same pass.
//
// Each pair (x_a, x_b) of the first `rot` elements of a head row turns by its token's angle:
//   y_a = x_a cos - x_b sin,  y_b = x_b cos + x_a sin   (cos and sin times `factor`)
// where pair p is (2p, 2p + 1) (interleaved) or (p, p + rot/2) (halves).  With weights, x is
// first normalised: x * r * gamma * out_scale, r = 1 / sqrt(mean(x^2) + eps).  All in fp32,
// rounded once when stored.  The angle sum_a pos_a * freq_a is formed in 64 bits and reduced to
// a fraction of a turn before the fp32 sine and cosine: at position 10^6 a fp32 angle has lost
// all but a few bits of its fraction.
//
// One pass over the heads; HBM bounds it.  rope_kernel is the form for head rows of whole
// 16-byte vectors (D and rot multiples of 16, 16-byte spacing): a warp takes one token, computes
// the token's cos/sin once, and every lane keeps the 8 pairs it needs of them -- the same ones
// for every head -- in registers while the token's heads stream by, 16 elements a lane.  A lane
// holds both elements of its pairs in either layout, so the rotation needs no exchange; the norm
// is one shuffle reduction over a row's lanes.  Loads run ahead through a small cp.async ring per
// warp, across heads and tokens, so the angles' latency and the stores hide behind them (plain
// register loads, four rows at a time, took 73 us where this took 61).  Frequencies and weights
// sit in shared memory.  Measured on a B200: 44160 tokens x 16 heads of 128, three axes, 60 us
// (6.0 TB/s, 92% of the measured copy rate); norm + rotation + re-partition of Q, K and V of the
// same size 180 us (6.0 TB/s, 92%).  rope_rows_kernel takes every other shape, an element at a time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "api_common.h"
#include "kernels.h"
#include "norm_math.cuh"
#include "rope.h"
#include "sm100_ptx.cuh"

namespace cpattn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store(float* p, float x) { *p = x; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// (cos, sin) * factor of an angle in radians.
__device__ __forceinline__ float2 turn_by(double angle, float factor) {
  angle *= 0.15915494309189533577;  // 1 / (2 pi): whole turns drop out exactly
  angle -= rint(angle);
  float s, co;
  sincospif(2.0f * float(angle), &s, &co);
  return make_float2(co * factor, s * factor);
}

// (cos, sin) * factor of pair p at position row `pr`.
__device__ __forceinline__ float2 pair_angle(const RopeCall& c, int pr, int p) {
  double angle = 0.0;
  for (int a = 0; a < c.n_axes; ++a)
    angle = fma(double(c.pos[(long long)pr * c.n_axes + a]), c.freq[(long long)a * (c.rot / 2) + p], angle);
  return turn_by(angle, c.factor);
}

// One warp per head row, one element at a time: any D <= 256 and any even rot <= D.  A block
// takes a few tokens, computes their cos/sin once into shared memory, and its warps take the
// (token, head) rows.
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
        const float r = row_factor(a);
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

// ------------------------------------------------------------------ vector form
constexpr int kWarpsPerBlock = kThreads / 32;
constexpr int kBlocksPerSm = 2;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// 8 consecutive elements of a row, kSlots 16-byte slots each; a warp keeps kStages - 1 steps of loads
// in flight (2 blocks x 8 warps x 3 KB per SM in bf16; 2 and 6 stages measured 222 and 202 us where
// 4 take 180, on the 44160-token norm + re-partition of Q, K and V).  `fetch` copies them to this lane's 16-byte slots of a stage (32
// lanes apart), `load` takes them from there.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  static constexpr int kSlots = 1;
  static constexpr int kStages = 4;
  uint4 v;
  static __device__ __forceinline__ void fetch(uint32_t slot, const __nv_bfloat16* p) { cp_async16(slot, p); }
  __device__ __forceinline__ void load(const uint8_t* slot) { v = *reinterpret_cast<const uint4*>(slot); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)  // bf16 -> fp32 is exact
      f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  __device__ __forceinline__ void set(const float2 (&f)[4]) {
    v = make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                   pack_bf16x2(f[3].x, f[3].y));
  }
};
template <>
struct Vec8<float> {
  static constexpr int kSlots = 2;
  static constexpr int kStages = 3;
  float4 a, b;
  static __device__ __forceinline__ void fetch(uint32_t slot, const float* p) {
    cp_async16(slot, p);
    cp_async16(slot + 512, p + 4);
  }
  __device__ __forceinline__ void load(const uint8_t* slot) {
    a = *reinterpret_cast<const float4*>(slot);
    b = *reinterpret_cast<const float4*>(slot + 512);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + 4) = b;
  }
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
  }
  __device__ __forceinline__ void set(const float2 (&f)[4]) {
    a = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    b = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  }
};

// A warp takes (token, part): one of 2^parts_log2 parts of the token's heads.  A row's D/16 lanes (padded
// to `lanes`, a power of two) hold two 8-element vectors each: lane l < rot/16 the vectors l and
// l + rot/16 of the rotated elements, the others two of the rest.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) rope_kernel(const __grid_constant__ RopeCall c, int lanes_log2,
                                                           int parts_log2) {
  __shared__ __align__(16) float2 cs_sh[kWarpsPerBlock][kRopeMaxD / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float2* cs = cs_sh[warp];
  const int D = c.D, half = c.rot / 2;
  const int L = D / 16, nr = c.rot / 16;
  const int rows_per_warp = 32 >> lanes_log2;
  const int l = lane & ((1 << lanes_log2) - 1), sub = lane >> lanes_log2;
  const bool live = l < L, turns = l < nr;
  const int va = 8 * (turns ? l : l + nr);                 // element of the first vector
  const int vb = turns ? va + half : va + 8 * (L - nr);    // and of the second
  const float inv_d = 1.0f / float(D);

  griddep_wait();
  griddep_release();

  // weights of the normalised tensors (at most the first two)
  __shared__ __align__(16) float gamma_sh[2][kRopeMaxD];
  __shared__ double freq_sh[4 * kRopeMaxD / 2];
  for (int e = threadIdx.x; e < c.n_axes * half; e += kThreads) freq_sh[e] = c.freq[e];
#pragma unroll
  for (int t = 0; t < 2; ++t)
    if (t < c.n_tensors && c.t[t].gamma != nullptr && int(threadIdx.x) < D) gamma_sh[t][threadIdx.x] = c.t[t].gamma[threadIdx.x];
  __syncthreads();

  const int parts = 1 << parts_log2;
  const int n_items = c.tokens * parts;  // the launcher keeps it below 2^31 less the grid's warps
  const int n_warps = int(gridDim.x) * kWarpsPerBlock;
  const int first = int(blockIdx.x) * kWarpsPerBlock + warp;

  // Loads run kStages - 1 steps (of one warp-load of rows) ahead, over tensors and tokens alike;
  // a lane reads back only what it copied itself, so a stage needs no barrier.
  extern __shared__ __align__(16) uint8_t ring[];
  using V = Vec8<T>;
  constexpr int kStageBytes = 2 * V::kSlots * 512, kStages = V::kStages;
  constexpr int kRingBytes = kStages * kStageBytes;
  uint8_t* slots = ring + warp * kRingBytes + lane * 16;
  const uint32_t slots_u32 = smem_u32(slots);
  int f_item = first, f_tensor = 0;  // the next step to fetch: item, tensor, first head
  int f_part = first & (parts - 1), f_head = 0, f_end = 0;
  const T* f_src = nullptr;
  auto heads_of = [&](int ti, int part, int& h_begin, int& h_end) {
    const int heads = c.t[ti].heads;
    h_begin = heads * part >> parts_log2;
    h_end = heads * (part + 1) >> parts_log2;
  };
  auto open = [&]() {  // f_item's token and tensor
    heads_of(f_tensor, f_part, f_head, f_end);
    const int token = f_item >> parts_log2;
    f_src = static_cast<const T*>(c.t[f_tensor].src) + (long long)token * c.t[f_tensor].src_stride;
  };
  auto settle = [&]() {  // on to the next tensor or item that has a head left
    while (f_head >= f_end) {
      if (++f_tensor >= c.n_tensors) {
        f_tensor = 0;
        f_item += n_warps;
        if (f_item >= n_items) return;
        f_part = f_item & (parts - 1);
      }
      open();
    }
  };
  auto fetch = [&](int stage) {
    if (f_item < n_items) {
      const int h = f_head + sub;
      if (live && h < f_end) {
        V::fetch(slots_u32 + stage * kStageBytes, f_src + h * D + va);
        V::fetch(slots_u32 + stage * kStageBytes + kStageBytes / 2, f_src + h * D + vb);
      }
      f_head += rows_per_warp;
      settle();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (f_item < n_items) {
    open();
    settle();
  }
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);

  // lane a holds axis a's position of the next item, loaded one item ahead
  auto position = [&](int item) {
    const int row = (item >> parts_log2) % c.pos_rows;
    return lane < c.n_axes ? c.pos[(long long)row * c.n_axes + lane] : 0;
  };
  int next_pos = first < n_items ? position(first) : 0;
  int stage = 0;
  for (int item = first; item < n_items; item += n_warps) {
    const int token = item >> parts_log2, part = item & (parts - 1);
    const int pos = next_pos;
    if (item + n_warps < n_items) next_pos = position(item + n_warps);
    __syncwarp();  // the previous token's angles are read no more
    // two pairs a lane at a time: the chain of one (64-bit products, conversions, sine and cosine) is long
    int p0 = 0;
    for (; p0 + 32 < half; p0 += 64) {
      const int pa = p0 + lane, pb = min(pa + 32, half - 1);
      double xa = 0.0, xb = 0.0;
      for (int a = 0; a < c.n_axes; ++a) {
        const double at = __shfl_sync(0xffffffffu, pos, a);
        xa = fma(at, freq_sh[a * half + pa], xa);
        xb = fma(at, freq_sh[a * half + pb], xb);
      }
      const float2 ca = turn_by(xa, c.factor), cb = turn_by(xb, c.factor);
      cs[pa] = ca;
      cs[pb] = cb;
    }
    if (p0 < half) {
      const int p = min(p0 + lane, half - 1);
      double x = 0.0;
      for (int a = 0; a < c.n_axes; ++a) x = fma(double(__shfl_sync(0xffffffffu, pos, a)), freq_sh[a * half + p], x);
      cs[p] = turn_by(x, c.factor);
    }
    __syncwarp();
    // cos and sin of this lane's pairs: 8 l + i (halves), or 4 (va / 8) + i and 4 (vb / 8) + i
    float2 w[8];
    if (turns) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = cs[kInterleaved ? (i < 4 ? va / 2 + i : vb / 2 + i - 4) : va + i];
    }
    for (int ti = 0; ti < c.n_tensors; ++ti) {
      const RopeTensor& t = c.t[ti];
      T* dst = static_cast<T*>(t.dst) + (long long)token * t.dst_stride;
      const bool norm = t.gamma != nullptr, rotate = t.rotate;
      int h0, h_end;
      heads_of(ti, part, h0, h_end);
      for (; h0 < h_end; h0 += rows_per_warp) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        V xa, xb;
        xa.load(slots + stage * kStageBytes);
        xb.load(slots + stage * kStageBytes + kStageBytes / 2);
        fetch(stage == 0 ? kStages - 1 : stage - 1);  // the stage read in the step before
        stage = stage + 1 == kStages ? 0 : stage + 1;
        const int h = h0 + sub;
        const bool on = live && h < h_end;
        if (norm || rotate) {  // otherwise the rows only move, bit for bit
          float2 a[4], b[4];
          xa.get(a);
          xb.get(b);
          if (norm) {
            float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) s2 = ffma2(b[i], b[i], ffma2(a[i], a[i], s2));
            float ss = on ? s2.x + s2.y : 0.f;
#pragma unroll
            for (int o = 1; o < 16; o <<= 1)
              if (o < (1 << lanes_log2)) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float mean = ss * inv_d + c.eps;
            const float r = row_factor(mean);
            const float2 r2 = make_float2(r, r), os = make_float2(c.out_scale, c.out_scale);
            const float4* ga = reinterpret_cast<const float4*>(&gamma_sh[ti & 1][live ? va : 0]);
            const float4* gb = reinterpret_cast<const float4*>(&gamma_sh[ti & 1][live ? vb : 0]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float4 p = ga[i], q = gb[i];
              a[2 * i] = fmul2(fmul2(a[2 * i], r2), make_float2(p.x, p.y));
              a[2 * i + 1] = fmul2(fmul2(a[2 * i + 1], r2), make_float2(p.z, p.w));
              b[2 * i] = fmul2(fmul2(b[2 * i], r2), make_float2(q.x, q.y));
              b[2 * i + 1] = fmul2(fmul2(b[2 * i + 1], r2), make_float2(q.z, q.w));
            }
            if (c.out_scale != 1.f) {  // (times 1 changes nothing)
#pragma unroll
              for (int i = 0; i < 4; ++i) a[i] = fmul2(a[i], os), b[i] = fmul2(b[i], os);
            }
          }
          if (turns && rotate) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if constexpr (kInterleaved) {  // (x0 c - x1 s, x1 c + x0 s)
                const float2 x = a[i], y = b[i], wa = w[i], wb = w[4 + i];
                a[i] = ffma2(x, make_float2(wa.x, wa.x), fmul2(make_float2(x.y, x.x), make_float2(-wa.y, wa.y)));
                b[i] = ffma2(y, make_float2(wb.x, wb.x), fmul2(make_float2(y.y, y.x), make_float2(-wb.y, wb.y)));
              } else {  // pairs 2i and 2i + 1: a cos - b sin, b cos + a sin
                const float2 x = a[i], y = b[i], w0 = w[2 * i], w1 = w[2 * i + 1];
                a[i] = make_float2(fmaf(x.x, w0.x, -(y.x * w0.y)), fmaf(x.y, w1.x, -(y.y * w1.y)));
                b[i] = make_float2(fmaf(y.x, w0.x, x.x * w0.y), fmaf(y.y, w1.x, x.y * w1.y));
              }
            }
          }
          xa.set(a);
          xb.set(b);
        }
        if (on) {
          const int g = t.group_magic == 0 ? h : int(__umulhi(unsigned(h), t.group_magic));  // h / group
          T* d = dst + g * t.group_stride + (long long)(h - g * t.group) * D;
          xa.store(d + va);
          xb.store(d + vb);
        }
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename T>
cudaError_t launch_vector(const RopeCall& c, int max_heads, cudaStream_t stream) {
  auto kernel = c.interleaved ? rope_kernel<T, true> : rope_kernel<T, false>;
  int lanes_log2 = 0;
  while ((1 << lanes_log2) < c.D / 16) ++lanes_log2;
  const int rows_per_warp = 32 >> lanes_log2;
  // Warps that share a token's heads, each with its own angles: as many as give the fewest steps to the
  // warp with the most, an item's angles counted as 2.5 steps.  Measured, parts 1 / 2 / 4: 1000 tokens
  // x 32 heads - / 6.1 / 9.1 us, 2000 10.2 / 11.6 / 14, 3000 17.5 / 16.2 / 23, 5000 22.4 / 22.8 / 34, 8000
  // 31.5 / 32.3 / 51.
  const long long warps = (long long)sm_count() * kBlocksPerSm * kWarpsPerBlock;
  int parts_log2 = 0;
  double least = 0.0;
  for (int p = 0; p == 0 || rows_per_warp << (p - 1) < max_heads; ++p) {
    const long long items = (long long)c.tokens << p;
    if (p > 0 && items > 1 << 30) break;
    double steps = 2.5;
    for (int t = 0; t < c.n_tensors; ++t) {
      const int heads = (c.t[t].heads + (1 << p) - 1) >> p;
      steps += (heads + rows_per_warp - 1) / rows_per_warp;
    }
    const double cost = double((items + warps - 1) / warps) * steps;
    if (p == 0 || cost < least) least = cost, parts_log2 = p;
  }
  const long long blocks = (((long long)c.tokens << parts_log2) + kWarpsPerBlock - 1) / kWarpsPerBlock;
  const long long cap = (long long)sm_count() * kBlocksPerSm;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks < cap ? blocks : cap));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kWarpsPerBlock * Vec8<T>::kStages * 2 * Vec8<T>::kSlots * 512;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static SmemOptIn opt_in[2];
  const cudaError_t e = opt_in[c.interleaved](reinterpret_cast<const void*>(kernel), int(cfg.dynamicSmemBytes));
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, kernel, c, lanes_log2, parts_log2);
}

// Can the vector form take this call?  Whole vectors, every row on 16 bytes.
bool vector_form(const RopeCall& c) {
  if (c.D % 16 != 0 || c.rot % 16 != 0) return false;
  const int vec = c.f32 ? 4 : 8;
  for (int i = 0; i < c.n_tensors; ++i)
    if (c.t[i].src_stride % vec != 0 || c.t[i].dst_stride % vec != 0 || c.t[i].group_stride % vec != 0) return false;
  return true;
}

}  // namespace

cudaError_t launch_rope(const RopeCall& call, cudaStream_t stream) {
  RopeCall c = call;
  int max_heads = 0;
  for (int i = 0; i < c.n_tensors; ++i) {
    RopeTensor& t = c.t[i];
    // h / group = umulhi(h, ceil(2^32 / group)) for h, group < 2^16; group 1 has no 32-bit form
    t.group_magic = t.group == 1 ? 0u : unsigned(((1ULL << 32) + t.group - 1) / t.group);
    if (t.heads > max_heads) max_heads = t.heads;
  }
  if (vector_form(c))
    return c.f32 ? launch_vector<float>(c, max_heads, stream) : launch_vector<__nv_bfloat16>(c, max_heads, stream);
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
