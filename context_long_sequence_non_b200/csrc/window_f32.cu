// window_f32.cu -- windowed attention and its single-token form with fp32 inputs, on the CUDA cores.
//
// A block takes 8, 32 or 48 (token, head) rows of one key head and walks the keys that some row of
// them sees -- early (sink) keys, then the window, as one list -- 64 at a time: S = Q K^T, the online
// softmax in base 2 and O += P V, all in fp32.  (The tensor cores take fp32 digits only in parts, such as
// three bf16 numbers an operand and six products for one; that form was not built or measured.)
// Keys of the list that a row does not see weigh exactly 0; keys outside the list are
// never read.  D is padded to 64, 128 or 256 with zeros.
//
// Layout.  A warp holds R rows and a lane two of the 64 keys of S and D / 32 columns of O.  The
// shared-memory port bounds it: a 16-byte read costs 4 cycles of it when the lanes read different
// keys, 1 when they read the same row of Q or P, so four columns of S cost R + 8 cycles for 32 R
// FMAs a lane, four keys of O R + 16.  (A lane grid of 2 x 16, 4 rows a thread, costs 20 for 64:
// causal 2000 x 8 heads 351 us against 289, 3000 x 8 340 against 316.)  K and V have one buffer each
// and still arrive behind the arithmetic: the next K is copied during the softmax and P V, the next
// V during the next S.  Two blocks fit an SM up to D = 128.
//
// Heads that share a key head are rows of the same block, so their keys are copied once: 16
// sequences x 32 heads on 8, one token, 60 us against 273.
//
// Split.  A cluster of up to 8 blocks shares the key list of one row tile where the tiles alone
// leave SMs idle; the parts (m, l, O) are folded through distributed shared memory in a fixed order.
// One token x 8 heads, 8192 keys of 128: 36 us (827 with neither the split nor one-row warps).
// Measured besides: 3000 x 8 heads of 128, 800 keys before and 100 after, 316 us = 31 TFLOP/s of visible
// products (its form, six rows a warp at D = 128, spills 8 bytes); 16 sequences x 32 heads on 8, one
// token, 2048 keys, 65 us = 4.2 TB/s; one token x 8 heads, 8192 keys, 1.9 TB/s: 64 blocks of 16 chunks of
// 64 keys, each chunk's copy, S, softmax and P V one behind another.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "api_common.h"
#include "kernels.h"
#include "sm100_ptx.cuh"
#include "window.h"

namespace cpattn {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 64;
constexpr int kMaxCluster = 8;
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

// R rows a warp, 8 R a block.
template <int DP, int R>
struct Tile {
  static constexpr int kRows = kWarps * R;
  static constexpr int kStrideK = DP + 4;  // the 32 keys of a read fall in different banks
  static constexpr int kOffK = kRows * DP;
  static constexpr int kOffV = kOffK + kKeys * kStrideK;
  static constexpr int kOffP = kOffV + kKeys * DP;
  static constexpr int kPartO = kRows * DP;  // a part's O, and behind it its m and l, where K was
  static_assert(kPartO + 2 * kRows <= kKeys * kStrideK);
  static constexpr int kSmem = (kOffP + kRows * kKeys) * 4;
};

template <int DP, int R>
__global__ void __launch_bounds__(kThreads, DP <= 128 ? 2 : 1) window_f32_kernel(const __grid_constant__ WindowCall c, int n_tiles, int n_group,
                                                              float scale_log2, bool vec) {
  using T = Tile<DP, R>;
  constexpr int kPairs = DP / 64, kRows = T::kRows;  // columns of a lane, in pairs
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;
  float* sk = sm + T::kOffK;
  float* sv = sm + T::kOffV;
  const int lane = threadIdx.x & 31;
  const int row0 = R * __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);  // the warp's rows
  float* sp = sm + T::kOffP + row0 * kKeys;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = int(cluster.block_rank()), n_ranks = int(cluster.num_blocks());
  // tiles with the most keys first, of all heads side by side: the grid ends on short ones
  const unsigned n_heads = unsigned(c.Hkv) * unsigned(c.B), item = blockIdx.x / unsigned(n_ranks);
  const int tile = n_tiles - 1 - int(item / n_heads);
  const int bh = int(item % n_heads);
  const int b = bh / c.Hkv, kvh = bh - b * c.Hkv;
  // row r of the block is token (q0 + r) / G, head kvh G + (q0 + r) % G
  const int G = n_group, q0 = tile * kRows, n_rows = min(kRows, c.Sq * G - q0);
  auto token = [&](int r) { return G == 1 ? q0 + r : int(unsigned(q0 + r) / unsigned(G)); };

  griddep_wait();
  griddep_release();

  const int len = sequence_length(c, b);
  const int off = c.from_end ? len - c.Sq : c.off;
  int early, lo, n;  // keys that some row sees: [0, early), then [lo, lo + n - early)
  int first;         // this block's share of that list: [first, n)
  {
    const KeyRange a = visible_keys(off + token(0), c.left, c.right, c.sinks, len);
    const KeyRange z = visible_keys(off + token(n_rows - 1), c.left, c.right, c.sinks, len);
    lo = a.lo < z.hi ? a.lo : z.hi;
    early = c.sinks < lo ? c.sinks : lo;
    n = early + (z.hi - lo);
    const int share = ((n + kKeys - 1) / kKeys + n_ranks - 1) / n_ranks * kKeys;
    first = min(n, rank * share);
    n = min(n, first + share);
  }
  const float* qp = static_cast<const float*>(c.q) + (long long)b * c.Sq * c.q_stride + (long long)kvh * G * c.D;
  const float* kp = static_cast<const float*>(c.k) + (long long)b * c.Skv * c.k_stride + (long long)kvh * c.D;
  const float* vp = static_cast<const float*>(c.v) + (long long)b * c.Skv * c.v_stride + (long long)kvh * c.D;

  // copy rows 0 .. n_live - 1 of `dst` from base + row(r) in the background, zeros elsewhere: one
  // cp.async group, of 16 bytes where every row allows it, else of 4
  auto fetch = [&](float* dst, int pitch, int rows, int n_live, const float* base, auto row) {
    if (vec) {
      for (int e = threadIdx.x; e < rows * (DP / 4); e += kThreads) {
        const int r = e / (DP / 4), d = 4 * (e % (DP / 4));
        const bool live = r < n_live && d < c.D;
        cp_async<16>(dst + r * pitch + d, live ? base + row(r) + d : base, live);
      }
    } else {
      for (int e = threadIdx.x; e < rows * DP; e += kThreads) {
        const int r = e / DP, d = e % DP;
        const bool live = r < n_live && d < c.D;
        cp_async<4>(dst + r * pitch + d, live ? base + row(r) + d : base, live);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto key_at = [&](int e) { return (long long)(e < early ? e : lo + (e - early)); };
  auto fetch_k = [&](int e0) {
    fetch(sk, T::kStrideK, kKeys, min(kKeys, n - e0), kp, [&](int r) { return key_at(e0 + r) * c.k_stride; });
  };
  auto fetch_v = [&](int e0) {
    fetch(sv, DP, kKeys, min(kKeys, n - e0), vp, [&](int r) { return key_at(e0 + r) * c.v_stride; });
  };
  fetch(sq, DP, kRows, n_rows, qp,
        [&](int r) { return token(r) * c.q_stride + (q0 + r - token(r) * G) * (long long)c.D; });
  if (first < n) {
    fetch_k(first);
    fetch_v(first);
  }

  const bool busy = row0 < n_rows;  // the warp has rows
  int pos[R];
#pragma unroll
  for (int i = 0; i < R; ++i) pos[i] = off + token(min(row0 + i, n_rows - 1));
  float m[R], l[R];
  float2 o[R][kPairs];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int g = 0; g < kPairs; ++g) o[i][g] = make_float2(0.f, 0.f);
  }

  for (int e0 = first; e0 < n; e0 += kKeys) {
    const int live = min(kKeys, n - e0);
    const bool more = e0 + kKeys < n;
    asm volatile("cp.async.wait_group 1;" ::: "memory");  // Q and these keys; their values may be under way
    __syncthreads();
    float2 s[R][2];
#pragma unroll
    for (int i = 0; i < R; ++i) s[i][0] = s[i][1] = make_float2(0.f, 0.f);
    if (busy) {
#pragma unroll 8
      for (int d = 0; d < DP; d += 4) {
        const float4 k0 = *reinterpret_cast<const float4*>(sk + lane * T::kStrideK + d);
        const float4 k1 = *reinterpret_cast<const float4*>(sk + (lane + 32) * T::kStrideK + d);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float4 q = *reinterpret_cast<const float4*>(sq + (row0 + i) * DP + d);
          s[i][0] = ffma2(make_float2(q.x, q.y), make_float2(k0.x, k0.y), s[i][0]);
          s[i][1] = ffma2(make_float2(q.x, q.y), make_float2(k1.x, k1.y), s[i][1]);
          s[i][0] = ffma2(make_float2(q.z, q.w), make_float2(k0.z, k0.w), s[i][0]);
          s[i][1] = ffma2(make_float2(q.z, q.w), make_float2(k1.z, k1.w), s[i][1]);
        }
      }
    }
    __syncthreads();  // K is read: the next keys' may come, while the softmax and P V run
    if (more) fetch_k(e0 + kKeys);
    else asm volatile("cp.async.commit_group;" ::: "memory");
    if (busy) {
      const int key[2] = {int(key_at(e0 + lane)), int(key_at(e0 + lane + 32))};
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const KeyRange see = visible_keys(pos[i], c.left, c.right, c.sinks, len);
        float x[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bool seen = lane + 32 * j < live && key[j] < see.hi && (key[j] >= see.lo || key[j] < see.early);
          x[j] = seen ? (s[i][j].x + s[i][j].y) * scale_log2 : -INFINITY;
        }
        float mx = fmaxf(x[0], x[1]);
#pragma unroll
        for (int y = 16; y > 0; y >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
        if (mx > m[i]) {  // the same for the whole warp
          const float a = ex2(m[i] - mx);
          m[i] = mx;
          l[i] *= a;
#pragma unroll
          for (int g = 0; g < kPairs; ++g) o[i][g].x *= a, o[i][g].y *= a;
        }
        const float ref = m[i] == -INFINITY ? 0.f : m[i];  // no key seen so far: every weight is 0
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float p = ex2(x[j] - ref);
          l[i] += p;
          sp[i * kKeys + lane + 32 * j] = p;
        }
      }
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");  // the values
    __syncthreads();  // (a row's weights are written and read by one warp)
    if (busy) {
#pragma unroll 4
      for (int j = 0; j < kKeys; j += 4) {
        float2 v[4][kPairs];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float* at = sv + (j + x) * DP;
          if constexpr (kPairs == 1) {
            v[x][0] = *reinterpret_cast<const float2*>(at + 2 * lane);
          } else {
#pragma unroll
            for (int g = 0; g < kPairs; g += 2) {
              const float4 y = *reinterpret_cast<const float4*>(at + 4 * lane + 64 * g);
              v[x][g] = make_float2(y.x, y.y), v[x][g + 1] = make_float2(y.z, y.w);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float4 p = *reinterpret_cast<const float4*>(sp + i * kKeys + j);
#pragma unroll
          for (int g = 0; g < kPairs; ++g) {
            o[i][g] = ffma2(make_float2(p.x, p.x), v[0][g], o[i][g]);
            o[i][g] = ffma2(make_float2(p.y, p.y), v[1][g], o[i][g]);
            o[i][g] = ffma2(make_float2(p.z, p.z), v[2][g], o[i][g]);
            o[i][g] = ffma2(make_float2(p.w, p.w), v[3][g], o[i][g]);
          }
        }
      }
    }
    if (more) {
      __syncthreads();  // V is read: the next one's copy runs beside the next S
      fetch_v(e0 + kKeys);
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);

  // column of a lane's pair g
  auto column = [&](int g) { return kPairs == 1 ? 2 * lane : 4 * lane + 128 * (g / 2) + 2 * (g % 2); };
  if (n_ranks > 1) {  // fold the parts; each block finishes every n_ranks-th row
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int g = 0; g < kPairs; ++g) *reinterpret_cast<float2*>(sk + (row0 + i) * DP + column(g)) = o[i][g];
      if (lane == 0) {
        sk[T::kPartO + row0 + i] = m[i];
        sk[T::kPartO + kRows + row0 + i] = l[i];
      }
    }
    cluster.sync();
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if ((row0 + i) % n_ranks != rank || row0 + i >= n_rows) continue;
      float mk[kMaxCluster], lk[kMaxCluster];
      float2 x[kMaxCluster][kPairs];
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {  // every remote read in flight at once
        mk[k] = -INFINITY;
        lk[k] = 0.f;
#pragma unroll
        for (int g = 0; g < kPairs; ++g) x[k][g] = make_float2(0.f, 0.f);
        if (k < n_ranks) {
          mk[k] = *cluster.map_shared_rank(sk + T::kPartO + row0 + i, k);
          lk[k] = *cluster.map_shared_rank(sk + T::kPartO + kRows + row0 + i, k);
#pragma unroll
          for (int g = 0; g < kPairs; ++g)
            x[k][g] = *cluster.map_shared_rank(reinterpret_cast<float2*>(sk + (row0 + i) * DP + column(g)), k);
        }
      }
      m[i] = mk[0];
#pragma unroll
      for (int k = 1; k < kMaxCluster; ++k) m[i] = fmaxf(m[i], mk[k]);
      l[i] = 0.f;
#pragma unroll
      for (int g = 0; g < kPairs; ++g) o[i][g] = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        const float w = lk[k] == 0.f ? 0.f : ex2(mk[k] - m[i]);  // 0: that block saw no key
        l[i] = fmaf(w, lk[k], l[i]);
#pragma unroll
        for (int g = 0; g < kPairs; ++g) o[i][g] = ffma2(make_float2(w, w), x[k][g], o[i][g]);
      }
    }
  }

#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = row0 + i;
    if (r >= n_rows || r % n_ranks != rank) continue;
    // No visible key: O = 0, LSE = -inf.  (Told by l, 1 or more with some: m is -inf for NaN scores too,
    // which the maximum drops, and their NaN l and O are the result.)
    const bool empty = l[i] == 0.f;
    const float inv = empty ? 0.f : 1.0f / l[i];
    const int t = token(r), h = kvh * G + (q0 + r - t * G);
    const long long at = (((long long)b * c.Sq + t) * c.H + h) * c.D;
#pragma unroll
    for (int g = 0; g < kPairs; ++g) {
      const float f[2] = {o[i][g].x * inv, o[i][g].y * inv};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int d = column(g) + x;
        if (d >= c.D) continue;
        if (c.out_f32) static_cast<float*>(c.out)[at + d] = f[x];
        else static_cast<__nv_bfloat16*>(c.out)[at + d] = __float2bfloat16_rn(f[x]);
      }
    }
    if (lane == 0 && c.lse != nullptr)
      c.lse[((long long)b * c.H + h) * c.Sq + t] = empty ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
  }
  if (n_ranks > 1) cluster.sync();  // no block leaves while another reads its shared memory
}

template <int DP, int R>
cudaError_t launch(const WindowCall& c, int n_ranks, cudaStream_t stream) {
  static SmemOptIn opt_in;
  cudaError_t e = opt_in(reinterpret_cast<const void*>(window_f32_kernel<DP, R>), Tile<DP, R>::kSmem);
  if (e != cudaSuccess) return e;
  const int n_tiles = int(((long long)c.Sq * (c.H / c.Hkv) + kWarps * R - 1) / (kWarps * R));
  const bool vec = c.D % 4 == 0 && c.q_stride % 4 == 0 && c.k_stride % 4 == 0 && c.v_stride % 4 == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(n_tiles) * unsigned(c.Hkv) * unsigned(c.B) * unsigned(n_ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Tile<DP, R>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(n_ranks);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, window_f32_kernel<DP, R>, c, n_tiles, c.H / c.Hkv,
                            float(double(c.scale) * 1.4426950408889634074), vec);
}

// Rows of a block and blocks of a row tile.  Six rows a warp read less per product than four, and
// pay where they fill the GPU's two places an SM one and a half times: 3000 x 8 heads 316 us against
// 339, 1500 x 16 272 against 302 (512 blocks), but causal 2000 x 8 378 against 294 (336).  Eight
// rows do not fit the registers of two blocks.  Where one block holds all rows of a key head, one row
// a warp: one token x 8 heads, 8192 keys, 36 us against 58.  More blocks share a tile while there is
// room on the GPU and a 64-key step for each: 1000 x 4 heads of 64, 300 keys, 22 us in two parts
// against 24; one token x 32 heads on 8, 1000 keys, 13 us in eight parts, 19 in four.
template <int DP>
cudaError_t launch_rows(const WindowCall& c, cudaStream_t stream) {
  const long long heads = (long long)c.Hkv * c.B, rows = (long long)c.H / c.Hkv * c.Sq, sms = sm_count();
  if constexpr (DP <= 128)
    if ((rows + 47) / 48 * heads >= 3 * sms) return launch<DP, 6>(c, 1, stream);
  const int tile = rows <= 8 ? 8 : 32;
  const long long blocks = (rows + tile - 1) / tile * heads, resident = DP <= 128 ? 2 * sms : sms;
  long long most = c.Skv;  // keys of a tile
  if (c.left >= 0 && c.right >= 0 && (long long)c.sinks + c.left + c.right + tile < most)
    most = (long long)c.sinks + c.left + c.right + tile;
  int n_ranks = 1;
  while (n_ranks < kMaxCluster && blocks * 2 * n_ranks <= resident && most > kKeys * n_ranks) n_ranks *= 2;
  return rows <= 8 ? launch<DP, 1>(c, n_ranks, stream) : launch<DP, 4>(c, n_ranks, stream);
}

}  // namespace

cudaError_t launch_window_f32(const WindowCall& c, cudaStream_t stream) {
  if (c.D <= 64) return launch_rows<64>(c, stream);
  if (c.D <= 128) return launch_rows<128>(c, stream);
  return launch_rows<256>(c, stream);
}

}  // namespace cpattn
