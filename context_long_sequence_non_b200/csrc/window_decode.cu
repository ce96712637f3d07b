// window_decode.cu -- the single-token form of the windowed attention: the last Sq tokens of each
// sequence against its key/value cache, bf16.
//
// The work is reading the visible keys and values once: at one token per sequence a cache row of
// 512 bytes meets 2 x 128 x (query heads per key head) products, so HBM bounds it and the
// products only have to stay out of the way.  The (token, head) rows that share a key head --
// Sq x H/Hkv of them -- are the M side of mma.m16n8k16 (16 rows a tile, padded): one read of K
// and V serves them all.  The tcgen05 forms need 64 or 128 rows of one operand, i.e. S^T with
// keys as rows and a softmax across TMEM lanes; the register fragments of the warp-level product
// feed the second product directly and cost a tenth of the time the loads take.
//
// Split.  A cluster of up to 8 CTAs x 4 warps shares one (sequence, key head, row tile): warp w of
// W takes every W-th chunk of the row tile's visible keys, with an online softmax of its own, and
// the partials (m, l, O) are folded in shared memory, then across the cluster through distributed
// shared memory -- one launch, no workspace, a fixed order of sums.  The cluster is as large as
// needed to occupy the GPU (decode_cluster below).
//
// Loads.  Each warp keeps kStages chunks of 16 keys in flight with 16-byte cp.async, 192 KB per SM
// (two CTAs of D = 128, four of D = 64), rows swizzled so that ldmatrix reads without bank
// conflicts.  Early (sink) keys and window keys form one list, so no chunk is spent on a boundary;
// rows that no query sees are never read, and the list's end is filled with zeros.
//
// Measured on a B200: 64 sequences x 32 heads on 8, 4100 keys at most, 122 us = 6.0 TB/s of K and V
// (92% of the measured copy rate; ncu counts 740 MB, the visible rows once); one sequence x 32 on 8
// over 1028 keys 5.5 us, all of it latency: two launches' overlap, one read, the fold; 8 sequences
// x 16 heads of 64, 4 tokens each, 12 to 13 us.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "api_common.h"
#include "kernels.h"
#include "sm100_ptx.cuh"
#include "window.h"

namespace cpattn {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kMaxCluster = 8;
constexpr int kRows = 16;  // (token, head) rows of a tile
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
struct Decode {
  static constexpr int kKeys = 16;  // keys of a chunk
  static constexpr int kStages = 3, kCtas = D == 128 ? 2 : 4;  // chunks in flight, CTAs per SM
  static constexpr int kRowBytes = D * 2;
  static constexpr int kVecs = D / 8;  // 16-byte vectors of a row
  static constexpr int kTile = kKeys * kRowBytes;
  static constexpr int kStage = 2 * kTile;  // K then V
  static constexpr int kLoads = kKeys * kVecs / 32;  // cp.async per lane and tensor
  static constexpr int kOStride = D + 4;  // floats; rows 16 bytes apart in the banks
  static constexpr int kPartial = kRows * kOStride * 4;
  static constexpr int kSmem = kWarps * kStages * kStage;
  static_assert(kSmem >= (kWarps + 1) * kPartial, "the partials reuse the stages");
};

// swizzled byte offset of vector v of row r
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int v) {
  return uint32_t(r * Decode<D>::kRowBytes + ((v ^ (r & 7)) << 4));
}

template <int D, bool kOutF32>
__global__ void __launch_bounds__(kWarps * 32, Decode<D>::kCtas)
    window_decode_kernel(const __grid_constant__ WindowCall c, int row_tiles, float scale_log2) {
  using T = Decode<D>;
  constexpr int kStages = T::kStages;
  constexpr int kN = T::kKeys / 8;  // 8-key column tiles of S
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ float part_m[kWarps][kRows], part_l[kWarps][kRows];
  __shared__ float cta_m[kRows], cta_l[kRows];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = int(cluster.block_rank()), n_ranks = int(cluster.num_blocks());
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = int(blockIdx.x) / n_ranks;  // (b, key head, row tile), row tile fastest
  const int rt = group % row_tiles;
  const int kvh = (group / row_tiles) % c.Hkv;
  const int b = group / row_tiles / c.Hkv;
  const int G = c.H / c.Hkv;
  const int row0 = rt * kRows;                    // first (token, head) row: token * G + head
  const int n_rows = min(kRows, G * c.Sq - row0);

  griddep_wait();

  const int len = sequence_length(c, b);
  const int off = len - c.Sq;
  // keys that some row of the tile sees, as one list: early ones, then [lo, hi)
  int early, lo, n;
  {
    const KeyRange a = visible_keys(off + row0 / G, c.left, c.right, c.sinks, len);
    const KeyRange z = visible_keys(off + (row0 + n_rows - 1) / G, c.left, c.right, c.sinks, len);
    lo = a.lo < z.hi ? a.lo : z.hi;
    early = c.sinks < lo ? c.sinks : lo;
    n = early + (z.hi - lo);
  }
  const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(c.k) + (long long)b * c.Skv * c.k_stride + (long long)kvh * D;
  const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(c.v) + (long long)b * c.Skv * c.v_stride + (long long)kvh * D;
  const uint32_t stages = smem_u32(smem) + uint32_t(warp * kStages * T::kStage);
  const int n_chunks = (n + T::kKeys - 1) / T::kKeys;
  const int step = kWarps * n_ranks;
  const int first = warp * n_ranks + rank;  // this warp's chunks: first, first + step, ...

  // start chunk `ch`'s copies into stage `st` (always one commit, so that the counts line up)
  auto fetch = [&](int ch, int st) {
    if (ch < n_chunks) {
      const uint32_t dst = stages + uint32_t(st * T::kStage);
#pragma unroll
      for (int i = 0; i < T::kLoads; ++i) {
        const int r = i * (32 / T::kVecs) + lane / T::kVecs, v = lane % T::kVecs;
        const int e = ch * T::kKeys + r;
        const bool live = e < n;
        const long long key = live ? (e < early ? e : lo + (e - early)) : 0;
        cp_async16(dst + swz<D>(r, v), kp + key * c.k_stride + v * 8, live);
        cp_async16(dst + T::kTile + swz<D>(r, v), vp + key * c.v_stride + v * 8, live);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(first + s * step, s);

  // Q fragments: thread's rows lane/4 and lane/4 + 8, columns 2 (lane % 4) + {0, 1} (+ 8)
  uint32_t qf[D / 16][4];
  KeyRange see[2];
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int r = lane / 4 + 8 * hh;
    const int row = row0 + (r < n_rows ? r : 0);
    const int i = row / G, g = row - i * G;
    see[hh] = visible_keys(off + i, c.left, c.right, c.sinks, len);
    const uint32_t* qp = reinterpret_cast<const uint32_t*>(
        static_cast<const __nv_bfloat16*>(c.q) + ((long long)b * c.Sq + i) * c.q_stride +
        ((long long)kvh * G + g) * D);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      qf[k][hh] = r < n_rows ? qp[k * 8 + (lane & 3)] : 0u;
      qf[k][2 + hh] = r < n_rows ? qp[k * 8 + 4 + (lane & 3)] : 0u;
    }
  }

  float o[D / 8][4];
#pragma unroll
  for (int t = 0; t < D / 8; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // base 2; l this thread's columns only

  int st = 0;
  for (int ch = first; ch < n_chunks; ch += step) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    {
      const int ahead = st + kStages - 1;
      fetch(ch + (kStages - 1) * step, ahead >= kStages ? ahead - kStages : ahead);
    }
    const uint32_t ks = stages + uint32_t(st * T::kStage), vs = ks + T::kTile;
    float s[kN][4];
#pragma unroll
    for (int t = 0; t < kN; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
    // S = Q K^T: matrices 0..3 of an ldmatrix are (keys 0-7, k 0-7), (0-7, 8-15), (8-15, 0-7),
    // (8-15, 8-15) of a 16-key, 16-column block
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
#pragma unroll
      for (int t = 0; t < kN; t += 2) {
        uint32_t kf[4];
        ldmatrix_x4(kf, ks + swz<D>(8 * t + (lane & 7) + 8 * (lane >> 4), 2 * k + ((lane >> 3) & 1)));
        mma16816(s[t], qf[k], kf[0], kf[1]);
        mma16816(s[t + 1], qf[k], kf[2], kf[3]);
      }
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int t = 0; t < kN; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at = ch * T::kKeys + 8 * t + 2 * (lane & 3) + (e & 1);
        const int key = at < early ? at : lo + (at - early);
        const KeyRange& r = see[e >> 1];
        const bool seen = at < n && key < r.hi && (key >= r.lo || key < r.early);
        s[t][e] = seen ? s[t][e] * scale_log2 : -INFINITY;
        mx[e >> 1] = fmaxf(mx[e >> 1], s[t][e]);
      }
    }
    float neg_m[2];
    bool grow = false;
    float alpha[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      mx[hh] = fmaxf(mx[hh], __shfl_xor_sync(0xffffffffu, mx[hh], 1));
      mx[hh] = fmaxf(mx[hh], __shfl_xor_sync(0xffffffffu, mx[hh], 2));
      const bool up = mx[hh] > m[hh];
      alpha[hh] = up ? ex2(m[hh] - mx[hh]) : 1.0f;
      if (up) m[hh] = mx[hh];
      grow |= up;
      neg_m[hh] = m[hh] == -INFINITY ? 0.f : -m[hh];
    }
    if (__any_sync(0xffffffffu, grow)) {
      l[0] *= alpha[0];
      l[1] *= alpha[1];
#pragma unroll
      for (int t = 0; t < D / 8; ++t) {
        o[t][0] *= alpha[0];
        o[t][1] *= alpha[0];
        o[t][2] *= alpha[1];
        o[t][3] *= alpha[1];
      }
    }
    uint32_t pf[kN / 2][4];  // P as the A operand: 16 keys a step
#pragma unroll
    for (int t = 0; t < kN; ++t) {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const float p0 = ex2(s[t][2 * hh] + neg_m[hh]), p1 = ex2(s[t][2 * hh + 1] + neg_m[hh]);
        l[hh] += p0 + p1;
        pf[t / 2][2 * (t & 1) + hh] = pack_bf16x2(p0, p1);  // bf16 weights; l keeps fp32
      }
    }
    // O += P V: V rows are keys, so the B operand comes transposed
#pragma unroll
    for (int kk = 0; kk < kN / 2; ++kk) {
#pragma unroll
      for (int t = 0; t < D / 8; t += 2) {
        uint32_t vf[4];
        ldmatrix_x4_trans(vf, vs + swz<D>(16 * kk + (lane & 15), t + (lane >> 4)));
        mma16816(o[t], pf[kk], vf[0], vf[1]);
        mma16816(o[t + 1], pf[kk], vf[2], vf[3]);
      }
    }
    st = st + 1 == kStages ? 0 : st + 1;
    __syncwarp();  // the stage is read before it is refilled
  }
  cp_async_wait<0>();
  // The next launch's blocks may take the places this one leaves from here on; let in at the start,
  // they crowded some SMs (8 sequences of 4 tokens, calls back to back: 15.1 us against 13.3).
  griddep_release();

  // ---- fold the warps' partials: m and l first, then O scaled to the block's maximum.  A row's keys are
  // told by l, 0 without any and 1 or more with some: m is -inf for NaN scores too, which the maximum
  // drops, and their NaN l and O are to reach the result
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
    l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
    if ((lane & 3) == 0) {
      part_m[warp][lane / 4 + 8 * hh] = m[hh];
      part_l[warp][lane / 4 + 8 * hh] = l[hh];
    }
  }
  __syncthreads();  // and every warp is done with the stages
  float* po = reinterpret_cast<float*>(smem) + warp * (T::kPartial / 4);
  float* co = reinterpret_cast<float*>(smem) + kWarps * (T::kPartial / 4);  // the block's sum
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int r = lane / 4 + 8 * hh;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_m[w][r]);
    const float w = l[hh] == 0.f ? 0.f : ex2(m[hh] - top);
    if (r < n_rows) {
#pragma unroll
      for (int t = 0; t < D / 8; ++t)
        *reinterpret_cast<float2*>(po + r * T::kOStride + t * 8 + 2 * (lane & 3)) =
            make_float2(o[t][2 * hh] * w, o[t][2 * hh + 1] * w);
    }
    if (warp == 0 && (lane & 3) == 0) {
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v)
        sum += part_l[v][r] == 0.f ? 0.f : part_l[v][r] * ex2(part_m[v][r] - top);
      cta_m[r] = top;
      cta_l[r] = sum;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < n_rows * (D / 4); e += kWarps * 32) {
    const int r = e / (D / 4), d = 4 * (e % (D / 4));
    const float* src = reinterpret_cast<const float*>(smem) + r * T::kOStride + d;
    float4 a = *reinterpret_cast<const float4*>(src);
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(src + w * (T::kPartial / 4));
      a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
    }
    *reinterpret_cast<float4*>(co + r * T::kOStride + d) = a;
  }
  if (n_ranks > 1) cluster.sync();
  else __syncthreads();

  // ---- fold the cluster: each block finishes every n_ranks-th group of four columns
  for (int e = int(threadIdx.x) * n_ranks + rank; e < n_rows * (D / 4); e += kWarps * 32 * n_ranks) {
    const int r = e / (D / 4), d = 4 * (e % (D / 4));
    float mk[kMaxCluster], lk[kMaxCluster];
    float4 xk[kMaxCluster];
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) {  // every remote read in flight at once
      mk[k] = -INFINITY;
      lk[k] = 0.f;
      xk[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < n_ranks) {
        mk[k] = *cluster.map_shared_rank(&cta_m[r], k);
        lk[k] = *cluster.map_shared_rank(&cta_l[r], k);
        xk[k] = *cluster.map_shared_rank(reinterpret_cast<float4*>(co + r * T::kOStride + d), k);
      }
    }
    float top = mk[0], sum = 0.f;
#pragma unroll
    for (int k = 1; k < kMaxCluster; ++k) top = fmaxf(top, mk[k]);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) {
      const float w = lk[k] == 0.f ? 0.f : ex2(mk[k] - top);  // 0: that block saw no key
      sum = fmaf(w, lk[k], sum);
      a.x = fmaf(w, xk[k].x, a.x), a.y = fmaf(w, xk[k].y, a.y), a.z = fmaf(w, xk[k].z, a.z), a.w = fmaf(w, xk[k].w, a.w);
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;  // no visible key: O = 0, LSE = -inf
    const int row = row0 + r, i = row / G, h = kvh * G + (row - i * G);
    const long long at = (((long long)b * c.Sq + i) * c.H + h) * D + d;
    if constexpr (kOutF32)
      *reinterpret_cast<float4*>(static_cast<float*>(c.out) + at) =
          make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(c.out) + at) =
          make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
    if (d == 0 && c.lse != nullptr)
      c.lse[((long long)b * c.H + h) * c.Sq + i] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
  if (n_ranks > 1) cluster.sync();  // no block leaves while another reads its shared memory
}

// CTAs that share a (sequence, key head, row tile): the count that minimises the modelled time.
// A CTA takes a fixed f (start, first loads, fold; more with a cluster to meet) and t for each
// chunk of its warps, t the chunk's latency or the share of an SM's bandwidth that its CTAs
// leave; when there is more than one wave of CTAs, half a CTA's time is lost at the end.
// Calibrated on a B200 (f = 3 or 4 us, t >= 0.6 us, 44 bytes per ns and SM): it picks the
// fastest of 1, 2, 4 and 8 on eight shapes from 8 to 1024 groups, where the wrong count costs
// from 10% to 9 times (1024 groups of 200 keys: 15 us with one CTA each, 67 us with eight).
template <int D>
int decode_cluster(long long groups, long long most_keys) {
  using T = Decode<D>;
  const double sms = sm_count();
  int best = 1;
  double best_t = 0;
  for (int n = 1; n <= kMaxCluster; n *= 2) {
    const double ctas = double(groups) * n;
    const double per_sm = ctas / sms < 1 ? 1 : (ctas / sms > T::kCtas ? T::kCtas : ctas / sms);
    const double share = per_sm * kWarps * T::kStage / 44e3;  // us per chunk at full bandwidth
    const long long chunks = (most_keys + T::kKeys - 1) / T::kKeys;
    const double own = double((chunks + kWarps * n - 1) / (kWarps * n));
    const double cta = (n > 1 ? 4.0 : 3.0) + own * (share > 0.6 ? share : 0.6);
    const double waves = ctas / (sms * T::kCtas);
    const double t = (waves <= 1 ? 1.0 : waves + 0.5) * cta;
    if (n == 1 || t < best_t) best = n, best_t = t;
  }
  return best;
}

template <int D, bool kOutF32>
cudaError_t launch(const WindowCall& c, cudaStream_t stream) {
  auto kernel = window_decode_kernel<D, kOutF32>;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in(reinterpret_cast<const void*>(kernel), Decode<D>::kSmem);
  if (e != cudaSuccess) return e;
  const int row_tiles = (c.H / c.Hkv * c.Sq + kRows - 1) / kRows;
  const long long groups = (long long)c.B * c.Hkv * row_tiles;
  long long most = c.Skv;
  if (c.left >= 0 && (long long)c.sinks + c.left + c.Sq < most) most = (long long)c.sinks + c.left + c.Sq;
  const int n = decode_cluster<D>(groups, most);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(groups * n));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = Decode<D>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(n);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, c, row_tiles, float(double(c.scale) * 1.4426950408889634074));
}

}  // namespace

cudaError_t launch_window_decode(const WindowCall& c, cudaStream_t stream) {
  if (c.D == 128) return c.out_f32 ? launch<128, true>(c, stream) : launch<128, false>(c, stream);
  return c.out_f32 ? launch<64, true>(c, stream) : launch<64, false>(c, stream);
}

}  // namespace cpattn
